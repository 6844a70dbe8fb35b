// ssm_bwd.hip -- the selective state space scan's backward.
//
// With e_t = dy_t z_t sigmoid(z_t), a_t = exp(s_t a) and r_t = a_t g_t h_{t-1}:
//   g_t = c_t e_t + a_{t+1} g_{t+1},
//   du = s sum_j g b + d e,  ds = u sum_j g b + sum_j a r,  ddt = ds softplus'(x),
//   dc = sum_i e h,  db = sum_i s u g,  da = sum_t s r,  dd = sum_t e u,
//   dz = dy (sum_j c h + d u) (z sigmoid(z))',  dh0 = a_0 g_0.
//
// Bound by the vector ALU, as the forward.  From the state that the forward kept before a chunk of 16 tokens the states of its later
// half are formed again into registers (64: two channels by four states by eight tokens a lane) and walked from their end, then those
// of its earlier half.  All 16 at once, with 16 states, would spill 136 registers; a state kept every eight tokens would double what a user keeps.
// Of more than 32 states all 16 tokens are held at once, since the sums over 16 lane groups take 16 tokens.
// Sums over states (du, ddt, dz) are in the lane but for steps over the lane groups, which four tokens share;
// sums over channels (db, dc) go through LDS: each token's eight values of a lane are summed eight lanes at a time, then over the
// workgroup's waves, and the workgroups' parts are added by a last launch, in a fixed order.
//
// 32768 x 2048 channels x 16 states in BF16, gated and packed: the segments from zero 270 us, the backward 1100 to 1170 us, the last launch 19 us.
// The vector ALU is busy for 77 and 70% of the first two's time.  What a gated wave holds, BF16 (FP32), and waves a SIMD:
//   states      registers  spilled   LDS of a workgroup  waves
//   up to 8     277 (308)  none      117 KB              one
//   9 to 16     256 (256)  27 (78)   73 KB               two
//   17 to 32    227 (234)  none      69 KB               two
//   33 to 64    313 (317)  none      91 KB               one
// 2 x 2048 x 2048 takes 170, 186, 295 and 802 us with 8, 16, 32 and 64 states (177, 208, 295 and 789), the launches before and after included.
#include "ssm_lay.hpp"

namespace lrs {
namespace {

// A chunk's values as they lie in memory.
template <class T, int NG>
struct Chunk {
    static constexpr int Q = Lay<NG>::Q;
    Pair<T> u[Q], dt[Q], z[Q], dy[Q];
    T b[NG], c[NG];
    Pair<float> h[4];
};
template <class T, int NG, bool GATE, bool SUM>
__device__ __forceinline__ void load_chunk(const SsmArgs& a, const Place& p, int chunk, Chunk<T, NG>& v) {
    const int64_t row0 = (int64_t)p.b * a.length + chunk * SSM_TOK;
    const int left = a.length - chunk * SSM_TOK, g = fresh_lane() / Lay<NG>::J;
    const char *u = rows_at<T>(a.u, row0, a.u_stride), *dt = rows_at<T>(a.dt, row0, a.dt_stride), *z = rows_at<T>(a.z, row0, a.z_stride),
            *dy = rows_at<T>(a.dy, row0, a.dy_stride);
    both_ways(a.per == 1, [&](auto one) {
        constexpr bool single = decltype(one)::value;
#pragma unroll
        for (int q = 0; q < Lay<NG>::Q; ++q) {
            const int r = min(q * NG + g, left - 1);
            if (!SUM) v.u[q] = Pair<T>::load(u, row_off<T>(r, a.u_stride, p.i), single);
            v.dt[q] = Pair<T>::load(dt, row_off<T>(r, a.dt_stride, p.i), single);
            v.dy[q] = Pair<T>::load(dy, row_off<T>(r, a.dy_stride, p.i), single);
            if (GATE) v.z[q] = Pair<T>::load(z, row_off<T>(r, a.z_stride, p.i), single);
        }
    });
    if (!SUM) load_group<T, NG>(a.b, a.b_stride, row0, left, p.gr, a.n, v.b);
    load_group<T, NG>(a.c, a.c_stride, row0, left, p.gr, a.n, v.c);
    if (!SUM) {
        const char* at = reinterpret_cast<const char*>(a.saved + ((int64_t)p.b * a.plan.chunks + chunk) * a.n * a.d);
#pragma unroll
        for (int s = 0; s < 4; ++s) v.h[s] = Pair<float>::load(at, state_off(a, min(4 * g + s, a.n - 1), p.i), a.per == 1);
    }
}

// A segment from its end with no cotangent from behind it: the product of its decays, and the cotangent that leaves it.
template <class T, int NG, bool GATE>
__global__ __launch_bounds__(256) void ssm_rev_kernel(const SsmArgs a) {
    using Y = Lay<NG>;
    constexpr int Q = Y::Q, J = Y::J;
    struct Wave {
        float4 se[SSM_TOK * J];  // s, e of two channels
        float4 c[SSM_TOK * NG];
    };
    __shared__ Wave waves[4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = a.plan.tiles * a.groups, segs = a.plan.segments - 1;
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit >= (int64_t)tiles * segs * a.batch) return;  // waves do not wait for each other
    const int tile = (int)(unit % tiles), seg = (int)(unit / tiles % segs) + 1, b = (int)(unit / tiles / segs);
    const Place p = place_of<NG>(a, tile % a.plan.tiles, tile / a.plan.tiles, seg, b);
    const int len = length_of(a, b);
    Wave& m = waves[wave];
    float A[2][4], G[2][4] = {};
    bool okn[4];
    load_rates(a, p, A, okn);
    const float2 bias = load_two(a, a.dt_bias, p);
    float2 total = make_float2(0.f, 0.f);
    bool anew = false;
    const int first = seg * a.plan.seg, last = min(first + a.plan.seg, a.plan.chunks);
    Chunk<T, NG> v;
    if (first < last) load_chunk<T, NG, GATE, true>(a, p, last - 1, v);
    for (int chunk = last - 1; chunk >= first; --chunk) {
        const uint32_t lane = fresh_lane();
        const int g = lane / J, j = lane % J;
        const int t0 = chunk * SSM_TOK, live = len - t0;
        const uint32_t resets = resets_of(a, b, t0);
        anew |= resets != 0;
        const auto stage = [&](auto mask, auto soft) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const float2 x = own(v.dt[q].get(), p);
                float2 e = own(v.dy[q].get(), p);
                float slope, s0 = x.x + bias.x, s1 = x.y + bias.y;
                if (decltype(soft)::value) s0 = softplus_of(s0, &slope), s1 = softplus_of(s1, &slope);
                if (GATE) {
                    const float2 z = own(v.z[q].get(), p);
                    e.x *= z.x * sigmoid_of(z.x), e.y *= z.y * sigmoid_of(z.y);
                }
                if (decltype(mask)::value) {  // padding may hold anything
                    const bool on = q * NG + g < live;
                    s0 = on ? s0 : 0.0f, s1 = on ? s1 : 0.0f;
                    e.x = on ? e.x : 0.0f, e.y = on ? e.y : 0.0f;
                }
                m.se[q * 64 + lane] = make_float4(s0, e.x, s1, e.y);
                total.x += s0, total.y += s1;
            }
            put_group<decltype(mask)::value, T, NG>(v.c, m.c, live, a.n);
        };
        both_ways(!whole_chunk<NG>(a, p.tile, live), [&](auto mask) { both_ways(a.softplus, [&](auto soft) { stage(mask, soft); }); });
        if (chunk > first) load_chunk<T, NG, GATE, true>(a, p, chunk - 1, v);
        wave_lds_sync();
        const auto walk = [&](auto starts) {
#pragma unroll
            for (int t = SSM_TOK - 1; t >= 0; --t) {
                const float4 x = m.se[t * J + j], C = m.c[t * NG + g];
                const float cs[4] = {C.x, C.y, C.z, C.w};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    G[0][s] = __builtin_amdgcn_exp2f(x.x * A[0][s]) * fmaf(cs[s], x.y, G[0][s]);
                    G[1][s] = __builtin_amdgcn_exp2f(x.z * A[1][s]) * fmaf(cs[s], x.w, G[1][s]);
                }
                if (decltype(starts)::value && (resets >> t & 1u)) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) G[0][s] = G[1][s] = 0.0f;
                }
                if (t % 2 == 0) __builtin_amdgcn_sched_barrier(0);
            }
        };
        both_ways(resets != 0, walk);
        wave_lds_sync();
    }
    put_segment<NG>(a, p, A, okn, total, anew, G);
}

// Waves of the workgroup hold channels of one group of b and c, side by side.
template <class T, int NG, int WAVES, bool GATE>
__global__ __launch_bounds__(64 * WAVES, 2) void ssm_bwd_kernel(const SsmArgs a) {
    using Y = Lay<NG>;
    constexpr int Q = Y::Q, J = Y::J, N4 = Y::N4, ROW = 68;  // a row of 64 lanes' values, padded
    constexpr int PART = NG == 16 ? 16 : 8, QP = PART / NG;   // tokens whose states are in registers at once
    // dy (z sigmoid(z))' of a token's channels, and once that is used, the sums of its dc and db over the wave's channels
    constexpr int PITCH = 2 * J > 8 * NG ? 2 * J : 8 * NG;
    struct Wave {
        float4 su[SSM_TOK * J];                                // s, s u of two channels
        float2 e[SSM_TOK * J], slope[SSM_TOK * J], u[SSM_TOK * J];  // e; softplus'; u
        float gate[SSM_TOK][PITCH];
        float4 b[SSM_TOK * NG], c[SSM_TOK * NG];
        float in[2][8 * ROW];                                  // a token's values of dc, db by lane
    };
    __shared__ Wave waves[WAVES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int blocks = a.plan.blocks * a.groups, segs = a.plan.segments;
    const int block = blockIdx.x % blocks, seg = blockIdx.x / blocks % segs, b = blockIdx.x / blocks / segs;
    const int gr = block / a.plan.blocks;
    const Place p = place_of<NG>(a, block % a.plan.blocks * WAVES + wave, gr, seg, b);
    const int len = length_of(a, b);
    Wave& m = waves[wave];

    float A[2][4], G[2][4], dA[2][4];
    bool okn[4];
    load_rates(a, p, A, okn);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            G[c][s] = dA[c][s] = 0.0f;
            if (!(c ? p.ok1 : p.ok0) || !okn[s]) continue;
            const int n = 4 * p.g + s;
            if (a.dh) G[c][s] = a.dh[((int64_t)b * a.d + p.c0 + c) * a.n + n];
        }
    through_segments(a, p, segs - 1, seg, -1, G);  // what those behind this one hand on
#pragma unroll
    for (int s = 0; s < 4; ++s) G[0][s] = p.ok0 && okn[s] ? G[0][s] : 0.0f, G[1][s] = p.ok1 && okn[s] ? G[1][s] : 0.0f;
    const float2 bias = load_two(a, a.dt_bias, p), skip = load_two(a, a.skip, p);
    float2 dskip = make_float2(0.f, 0.f), dbias = make_float2(0.f, 0.f);
    const int first = seg * a.plan.seg, last = min(first + a.plan.seg, a.plan.chunks);
    Chunk<T, NG> v;
    if (first < last) load_chunk<T, NG, GATE, false>(a, p, last - 1, v);
    for (int chunk = last - 1; chunk >= first; --chunk) {
        const uint32_t lane = fresh_lane();
        const int g = lane / J, j = lane % J;
        const int t0 = chunk * SSM_TOK, live = len - t0, left = a.length - t0;
        const int64_t row0 = (int64_t)b * a.length + t0;
        const uint32_t resets = resets_of(a, b, t0);
        float hin[2][4];
        const auto stage = [&](auto mask, auto soft) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float2 x = own(v.h[s].get(), p);
                const bool on = !decltype(mask)::value || okn[s];
                hin[0][s] = on ? x.x : 0.0f, hin[1][s] = on ? x.y : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const uint32_t at = q * 64 + lane;
                const float2 x = own(v.dt[q].get(), p), dy = own(v.dy[q].get(), p);
                float2 u = own(v.u[q].get(), p), slope = make_float2(1.f, 1.f), s = make_float2(x.x + bias.x, x.y + bias.y), e = dy;
                if (decltype(soft)::value) s.x = softplus_of(s.x, &slope.x), s.y = softplus_of(s.y, &slope.y);
                if (GATE) {
                    const float2 z = own(v.z[q].get(), p);
                    const float g0 = sigmoid_of(z.x), g1 = sigmoid_of(z.y), s0 = z.x * g0, s1 = z.y * g1;
                    e.x *= s0, e.y *= s1;
                    // (z sigmoid(z))' = sigmoid(z) + z sigmoid(z) (1 - sigmoid(z))
                    reinterpret_cast<float2*>(m.gate[q * NG + g])[j] = make_float2(dy.x * fmaf(s0, 1.0f - g0, g0), dy.y * fmaf(s1, 1.0f - g1, g1));
                }
                if (decltype(mask)::value) {  // padding may hold anything, and channels that do not exist add nothing to db and dc
                    const bool on = q * NG + g < live, on0 = on && p.ok0, on1 = on && p.ok1;
                    s.x = on ? s.x : 0.0f, s.y = on ? s.y : 0.0f;
                    u.x = on0 ? u.x : 0.0f, u.y = on1 ? u.y : 0.0f;
                    e.x = on0 ? e.x : 0.0f, e.y = on1 ? e.y : 0.0f;
                }
                m.u[at] = u;
                m.su[at] = make_float4(s.x, s.x * u.x, s.y, s.y * u.y);
                m.e[at] = e;
                m.slope[at] = slope;
            }
            put_group<decltype(mask)::value, T, NG>(v.b, m.b, live, a.n);
            put_group<decltype(mask)::value, T, NG>(v.c, m.c, live, a.n);
        };
        both_ways(!whole_chunk<NG>(a, p.tile, live), [&](auto mask) { both_ways(a.softplus, [&](auto soft) { stage(mask, soft); }); });
        if (chunk > first) load_chunk<T, NG, GATE, false>(a, p, chunk - 1, v);
        wave_lds_sync();

        // The states of PART tokens are formed again and walked from their end; first the later ones, from the state between them, which
        // a run through the earlier ones gives.  A chunk without a sequence's start, as most are, runs free of selects.
        const auto walk = [&](auto starts) {
            const auto begins = [&](int t) { return decltype(starts)::value && (resets >> t & 1u); };
            float mid[2][4];
            if constexpr (PART < SSM_TOK) {
#pragma unroll
                for (int s = 0; s < 4; ++s) mid[0][s] = hin[0][s], mid[1][s] = hin[1][s];
#pragma unroll
                for (int t = 0; t < PART; ++t) {
                    const float4 x = m.su[t * J + j], B = m.b[t * NG + g];
                    const float bs[4] = {B.x, B.y, B.z, B.w};
                    const bool start = begins(t);
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        mid[0][s] = fmaf(__builtin_amdgcn_exp2f(x.x * A[0][s]), start ? 0.0f : mid[0][s], x.y * bs[s]);
                        mid[1][s] = fmaf(__builtin_amdgcn_exp2f(x.z * A[1][s]), start ? 0.0f : mid[1][s], x.w * bs[s]);
                    }
                    if (t % 2) __builtin_amdgcn_sched_barrier(0);
                }
            }
            const auto part = [&](const int p0, const float (&from)[2][4]) {
                float h[PART][2][4];
#pragma unroll
                for (int q = 0; q < QP; ++q) {
                    float y0[NG], y1[NG];
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        const int k = q * NG + i, t = p0 + k;
                        const float4 x = m.su[t * J + j], B = m.b[t * NG + g];
                        const float bs[4] = {B.x, B.y, B.z, B.w};
                        const bool start = begins(t);
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const float before0 = start ? 0.0f : k ? h[k - 1][0][s] : from[0][s], before1 = start ? 0.0f : k ? h[k - 1][1][s] : from[1][s];
                            h[k][0][s] = fmaf(__builtin_amdgcn_exp2f(x.x * A[0][s]), before0, x.y * bs[s]);
                            h[k][1][s] = fmaf(__builtin_amdgcn_exp2f(x.z * A[1][s]), before1, x.w * bs[s]);
                        }
                        if (GATE) {
                            const float4 C = m.c[t * NG + g];
                            y0[i] = fmaf(C.w, h[k][0][3], fmaf(C.z, h[k][0][2], fmaf(C.y, h[k][0][1], C.x * h[k][0][0])));
                            y1[i] = fmaf(C.w, h[k][1][3], fmaf(C.z, h[k][1][2], fmaf(C.y, h[k][1][1], C.x * h[k][1][0])));
                        }
                        if (t % 2) __builtin_amdgcn_sched_barrier(0);
                    }
                    if (GATE) {  // the outputs before the gate, for its gradient
                        const int r = p0 + q * NG + g, at = (p0 / NG + q) * 64 + lane;
                        const bool on = r < live;
                        const float r0 = group_sum<NG>(y0), r1 = group_sum<NG>(y1);
                        const float2 w = reinterpret_cast<const float2*>(m.gate[r])[j], u = m.u[at];
                        const float2 dz = make_float2(on ? w.x * fmaf(skip.x, u.x, r0) : 0.0f, on ? w.y * fmaf(skip.y, u.y, r1) : 0.0f);
                        store_pair<T>(rows_at<T>(a.dz, row0, a.d), row_off<T>(r, a.d, p.c0), dz, r < left && p.ok0, r < left && p.ok1);
                    }
                }
                // dc and db of token t: lane r sums value r / 8 of lanes 8 (r % 8) and the seven behind it
                const auto sum_up = [&](int t) {
                    const float4* in = reinterpret_cast<const float4*>(m.in[t % 2] + (lane >> 3) * ROW + (lane & 7) * 8);
                    const float4 lo = in[0], hi = in[1];
                    float* to = m.gate[t] + (lane >> 3) * NG;
                    const float l = (lo.x + lo.y) + (lo.z + lo.w), u = (hi.x + hi.y) + (hi.z + hi.w);
                    if constexpr (NG == 16) {
                        to[2 * (lane & 7)] = l, to[2 * (lane & 7) + 1] = u;
                    } else {
                        float w = l + u;
                        if constexpr (NG <= 4) w += row_xor<1>(w);
                        if constexpr (NG <= 2) w += row_xor<2>(w);
                        if ((lane & 7) % (8 / NG) == 0) to[(lane & 7) * NG / 8] = w;
                    }
                };
#pragma unroll
                for (int q = QP - 1; q >= 0; --q) {
                    float gb0[NG], gb1[NG], ar0[NG], ar1[NG];
#pragma unroll
                    for (int i = NG - 1; i >= 0; --i) {
                        const int k = q * NG + i, t = p0 + k;
                        const float4 x = m.su[t * J + j], B = m.b[t * NG + g], C = m.c[t * NG + g];
                        const float2 e = m.e[t * J + j];
                        const float bs[4] = {B.x, B.y, B.z, B.w}, cs[4] = {C.x, C.y, C.z, C.w};
                        const bool start = begins(t);
                        float* in = m.in[t % 2] + lane;
                        // what the token behind this one left, while this one's is formed
                        if (k < PART - 1) sum_up(t + 1);
                        gb0[i] = gb1[i] = ar0[i] = ar1[i] = 0.0f;
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const float g0 = fmaf(cs[s], e.x, G[0][s]), g1 = fmaf(cs[s], e.y, G[1][s]);
                            in[s * ROW] = fmaf(e.x, h[k][0][s], e.y * h[k][1][s]);
                            in[(4 + s) * ROW] = fmaf(x.y, g0, x.w * g1);
                            gb0[i] = fmaf(g0, bs[s], gb0[i]), gb1[i] = fmaf(g1, bs[s], gb1[i]);
                            const float w0 = start ? 0.0f : __builtin_amdgcn_exp2f(x.x * A[0][s]) * g0;
                            const float w1 = start ? 0.0f : __builtin_amdgcn_exp2f(x.z * A[1][s]) * g1;
                            const float r0 = start ? 0.0f : w0 * (k ? h[k - 1][0][s] : from[0][s]), r1 = start ? 0.0f : w1 * (k ? h[k - 1][1][s] : from[1][s]);
                            ar0[i] = fmaf(r0, A[0][s], ar0[i]), ar1[i] = fmaf(r1, A[1][s], ar1[i]);
                            dA[0][s] = fmaf(x.x, r0, dA[0][s]), dA[1][s] = fmaf(x.z, r1, dA[1][s]);
                            G[0][s] = w0, G[1][s] = w1;
                            // here and now: moved to the chunk's end, these sums would keep all of its r in registers
                            asm volatile("" : "+v"(dA[0][s]), "+v"(dA[1][s]));
                        }
                        wave_lds_sync();
                    }
                    const int r = p0 + q * NG + g, at = (p0 / NG + q) * 64 + lane;
                    const float sb0 = group_sum<NG>(gb0), sb1 = group_sum<NG>(gb1);
                    const float sa0 = LN2 * group_sum<NG>(ar0), sa1 = LN2 * group_sum<NG>(ar1);  // A holds a log2 e
                    const float4 x = m.su[at];
                    const float2 e = m.e[at], slope = m.slope[at], u = m.u[at];
                    const bool on = r < live, in0 = r < left && p.ok0, in1 = r < left && p.ok1;
                    const float2 du = make_float2(on ? fmaf(x.x, sb0, skip.x * e.x) : 0.0f, on ? fmaf(x.z, sb1, skip.y * e.y) : 0.0f);
                    const float2 dd = make_float2(on ? fmaf(u.x, sb0, sa0) * slope.x : 0.0f, on ? fmaf(u.y, sb1, sa1) * slope.y : 0.0f);
                    dskip.x = fmaf(e.x, u.x, dskip.x), dskip.y = fmaf(e.y, u.y, dskip.y);
                    dbias.x += dd.x, dbias.y += dd.y;
                    const uint32_t off = row_off<T>(r, a.d, p.c0);
                    store_pair<T>(rows_at<T>(a.du, row0, a.d), off, du, in0, in1);
                    store_pair<T>(rows_at<T>(a.ddt, row0, a.d), off, dd, in0, in1);
                }
                sum_up(p0);
                wave_lds_sync();
            };
            if constexpr (PART < SSM_TOK) part(PART, mid);
            part(0, hin);
        };
        both_ways(resets != 0, walk);
        __syncthreads();
        for (int x = threadIdx.x; x < SSM_TOK * 8 * NG; x += 64 * WAVES) {
            const int n = x % N4, k = x / N4 % 2, t = x / (2 * N4), at = (k * 4 + n % 4) * NG + n / 4;
            float w = waves[0].gate[t][at];
#pragma unroll
            for (int i = 1; i < WAVES; ++i) w += waves[i].gate[t][at];
            if (t0 + t < a.length) a.part_bc[(((int64_t)block * a.batch + b) * a.length + t0 + t) * 2 * N4 + k * N4 + n] = w;
        }
        __syncthreads();
    }
    if (seg == 0 && a.dh0) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if ((c ? p.ok1 : p.ok0) && okn[s]) a.dh0[((int64_t)b * a.d + p.c0 + c) * a.n + 4 * p.g + s] = G[c][s];
    }
    const int64_t mine = (int64_t)b * segs + seg;
    char* at = reinterpret_cast<char*>(a.part_a + mine * a.n * a.d);
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (okn[s]) store_pair<float>(at, state_off(a, 4 * p.g + s, p.c0), make_float2(dA[0][s], dA[1][s]), p.ok0, p.ok1);
#pragma unroll
    for (int o = 32; o >= J; o >>= 1) {
        dskip.x += __shfl_xor(dskip.x, o), dskip.y += __shfl_xor(dskip.y, o);
        dbias.x += __shfl_xor(dbias.x, o), dbias.y += __shfl_xor(dbias.y, o);
    }
    if (p.g == 0) {
        char* pd = reinterpret_cast<char*>(a.part_d + mine * 2 * a.d);
        store_pair<float>(pd, state_off(a, 0, p.c0), dskip, p.ok0, p.ok1);
        store_pair<float>(pd, state_off(a, 1, p.c0), dbias, p.ok0, p.ok1);
    }
}

// Sums of the workgroups' parts, in a fixed order: db and dc over the channels' workgroups (FP32, as they are few), da, dskip
// and ddt_bias over rows and segments (FP64).  `x`: the first's number, or the second's.
template <class T>
__device__ __forceinline__ void join_narrow(const SsmArgs& a, int64_t x) {
    const int n4 = SSM_STATES * a.plan.ng;
    const int64_t rows = (int64_t)a.batch * a.length;
    if (x >= rows * a.groups * 2 * n4) return;
    const int n = (int)(x % n4), k = (int)(x / n4 % 2), gr = (int)(x / (2 * n4) / rows);
    const int64_t row = x / (2 * n4) % rows;
    if (n >= a.n) return;
    const float* at = a.part_bc + ((int64_t)gr * a.plan.blocks * rows + row) * 2 * n4 + k * n4 + n;
    float w = 0.0f;
    for (int i0 = 0; i0 < a.plan.blocks; i0 += 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = at[(int64_t)min(i0 + u, a.plan.blocks - 1) * rows * 2 * n4];
#pragma unroll
        for (int u = 0; u < 8; ++u) w += i0 + u < a.plan.blocks ? v[u] : 0.0f;
    }
    store_value(static_cast<T*>(k ? a.db : a.dc) + (row * a.groups + gr) * a.n + n, w);
}
__device__ __forceinline__ void join_channel(const SsmArgs& a, int64_t x) {
    const int i = (int)(x % a.d), n = (int)(x / a.d), parts = a.batch * a.plan.segments;
    if (n >= a.n + 2) return;
    const bool rate = n < a.n;
    const float* at = rate ? a.part_a + (int64_t)n * a.d + i : a.part_d + (int64_t)(n - a.n) * a.d + i;
    const int64_t step = rate ? (int64_t)a.n * a.d : 2 * (int64_t)a.d;
    double w = 0.0;
    for (int k0 = 0; k0 < parts; k0 += 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = at[min(k0 + u, parts - 1) * step];
#pragma unroll
        for (int u = 0; u < 8; ++u) w += k0 + u < parts ? (double)v[u] : 0.0;
    }
    float* out = rate ? a.da + (int64_t)i * a.n + n : n == a.n ? (a.dskip ? a.dskip + i : nullptr) : (a.ddt_bias ? a.ddt_bias + i : nullptr);
    if (out) *out = (float)w;
}
template <class T>
__global__ __launch_bounds__(256) void ssm_join_kernel(const SsmArgs a, int64_t first, int64_t narrow) {
    const int64_t w = first + blockIdx.x;
    if (w < narrow) join_narrow<T>(a, w * 256 + threadIdx.x);
    else join_channel(a, (w - narrow) * 256 + threadIdx.x);
}

template <class T, int NG, bool GATE>
void launch_gate(const SsmArgs& a, hipStream_t s) {
    constexpr int WAVES = 4;
    if (a.plan.segments > 1)
        LRS_LAUNCH(K_SSM_REV, (ssm_rev_kernel<T, NG, GATE>),
                   dim3((unsigned)ceil_div((int64_t)a.plan.tiles * a.groups * a.batch * (a.plan.segments - 1), 4)), dim3(256), 0, s, a);
    LRS_LAUNCH(K_SSM_BWD, (ssm_bwd_kernel<T, NG, WAVES, GATE>), dim3((unsigned)((int64_t)a.plan.blocks * a.groups * a.plan.segments * a.batch)),
               dim3(64 * WAVES), 0, s, a);
}
template <class T, int NG>
void launch_bwd(const SsmArgs& a, hipStream_t s) {
    if (a.z) launch_gate<T, NG, true>(a, s);
    else launch_gate<T, NG, false>(a, s);
}
template <class T>
void launch_bwd_any(const SsmArgs& a, hipStream_t s) {
    if (a.batch > 0) {
        switch (a.plan.ng) {
            case 2: launch_bwd<T, 2>(a, s); break;
            case 4: launch_bwd<T, 4>(a, s); break;
            case 8: launch_bwd<T, 8>(a, s); break;
            default: launch_bwd<T, 16>(a, s);
        }
    }
    const SsmJoin j = ssm_join(a.batch, a.length, a.d, a.n, a.groups, a.plan.ng);
    for (int64_t w = 0; w < j.all; w += j.grid)
        LRS_LAUNCH(K_SSM_JOIN, (ssm_join_kernel<T>), dim3((unsigned)std::min<int64_t>(j.grid, j.all - w)), dim3(256), 0, s, a, w, j.narrow);
}

}  // namespace

hipError_t launch_ssm_bwd(const SsmArgs& a, bool f32, hipStream_t s) {
    if (f32) launch_bwd_any<float>(a, s);
    else launch_bwd_any<uint16_t>(a, s);
    return hipGetLastError();
}

}  // namespace lrs
