// ssm_bwd.hip -- the selective state space scan's backward.
//
// With e_t = dy_t z_t sigmoid(z_t), a_t = exp(s_t a) and r_t = a_t g_t h_{t-1}:
//   g_t = c_t e_t + a_{t+1} g_{t+1},
//   du = s sum_j g b + d e,  ds = u sum_j g b + sum_j a r,  ddt = ds softplus'(x),
//   dc = sum_i e h,  db = sum_i s u g,  da = sum_t s r,  dd = sum_t e u,
//   dz = dy (sum_j c h + d u) (z sigmoid(z))',  dh0 = a_0 g_0.
//
// Bound by the vector ALU, as the forward.  From the state that the forward kept before a chunk its 16 states are formed
// again into registers (128 of them: two channels by four states by 16 tokens a lane), then the chunk is walked from its
// end.  Sums over states (du, ddt, dz) are in the lane but for steps over the lane groups, which four tokens share;
// sums over channels (db, dc) go through LDS: each token's eight values of a lane are summed eight lanes at a time, then over the
// workgroup's waves, and the workgroups' parts are added by a last launch, in a fixed order.
#include <type_traits>

#include "ssm_lay.hpp"

namespace lrs {
namespace {

// A chunk's values as they lie in memory.
template <class T, int NG>
struct Chunk {
    static constexpr int Q = Lay<NG>::Q;
    Pair<T> u[Q], dt[Q], z[Q], dy[Q];
    T b[NG], c[NG];
    float2 h[4];
};
template <class T, int NG, bool SUM>
__device__ __forceinline__ void load_chunk(const SsmArgs& a, const Place& p, int chunk, Chunk<T, NG>& v) {
    const int lane = threadIdx.x & 63, g = lane / Lay<NG>::J, t0 = chunk * SSM_TOK;
    const int64_t row0 = (int64_t)p.b * a.length;
#pragma unroll
    for (int q = 0; q < Lay<NG>::Q; ++q) {
        const int64_t row = row0 + min(t0 + q * NG + g, a.length - 1);
        if (!SUM) v.u[q] = Pair<T>::load(static_cast<const T*>(a.u) + row * a.u_stride, p.i, p.k, p.pair);
        v.dt[q] = Pair<T>::load(static_cast<const T*>(a.dt) + row * a.dt_stride, p.i, p.k, p.pair);
        v.dy[q] = Pair<T>::load(static_cast<const T*>(a.dy) + row * a.dy_stride, p.i, p.k, p.pair);
        if (a.z) v.z[q] = Pair<T>::load(static_cast<const T*>(a.z) + row * a.z_stride, p.i, p.k, p.pair);
    }
#pragma unroll
    for (int e = 0; e < NG; ++e) {
        const int x = e * 64 + lane, t = x / Lay<NG>::N4, n = min(x % Lay<NG>::N4, a.n - 1);
        const int64_t row = row0 + min(t0 + t, a.length - 1);
        if (!SUM) v.b[e] = static_cast<const T*>(a.b)[row * a.b_stride + p.gr * a.n + n];
        v.c[e] = static_cast<const T*>(a.c)[row * a.c_stride + p.gr * a.n + n];
    }
    if (!SUM) {
        const float* at = a.saved + ((int64_t)p.b * a.plan.chunks + chunk) * a.n * a.d;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const Pair<float> x = Pair<float>::load(at + (int64_t)min(4 * g + s, a.n - 1) * a.d, p.i, p.k, p.pair);
            v.h[s] = x.get();
        }
    }
}

// The decays' factors of a lane's states.
__device__ __forceinline__ void load_rates(const SsmArgs& a, const Place& p, int g, float (&A)[2][4], bool (&okn)[4]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int n = 4 * g + s;
        okn[s] = n < a.n;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            A[c][s] = (c ? p.ok1 : p.ok0) && okn[s] ? LOG2E * a.a[(int64_t)(p.c0 + c) * a.n + n] : 0.0f;
    }
}

// A segment from its end with no cotangent from behind it: the product of its decays, and the cotangent that leaves it.
template <class T, int NG>
__global__ __launch_bounds__(256) void ssm_rev_kernel(const SsmArgs a) {
    using Y = Lay<NG>;
    constexpr int Q = Y::Q, J = Y::J;
    __shared__ float4 s_dt[4][SSM_TOK * J];  // s, e of two channels
    __shared__ float4 s_c[4][SSM_TOK * NG];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane / J, j = lane % J;
    const int tiles = a.plan.tiles * a.groups, segs = a.plan.segments - 1;
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit >= (int64_t)tiles * segs * a.batch) return;  // waves do not wait for each other
    const int tile = (int)(unit % tiles), seg = (int)(unit / tiles % segs) + 1, b = (int)(unit / tiles / segs);
    const Place p = place_of<NG>(a, tile % a.plan.tiles, tile / a.plan.tiles, seg, b);
    const int len = length_of(a, b);
    float A[2][4], G[2][4] = {};
    bool okn[4];
    load_rates(a, p, g, A, okn);
    const float2 bias = a.dt_bias ? make_float2(a.dt_bias[p.i], a.dt_bias[p.k]) : make_float2(0.f, 0.f);
    float2 total = make_float2(0.f, 0.f);
    bool anew = false;
    const int first = seg * a.plan.seg, last = min(first + a.plan.seg, a.plan.chunks);
    Chunk<T, NG> v;
    if (first < last) load_chunk<T, NG, true>(a, p, last - 1, v);
    for (int chunk = last - 1; chunk >= first; --chunk) {
        const int t0 = chunk * SSM_TOK;
        const uint32_t resets = resets_of(a, b, t0, len);
        anew |= resets != 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int t = t0 + q * NG + g;
            const float2 x = v.dt[q].get();
            float2 e = v.dy[q].get();
            float slope, s0 = x.x + bias.x, s1 = x.y + bias.y;
            if (a.softplus) s0 = softplus_of(s0, &slope), s1 = softplus_of(s1, &slope);
            if (a.z) {
                const float2 z = v.z[q].get();
                e.x *= z.x * sigmoid_of(z.x), e.y *= z.y * sigmoid_of(z.y);
            }
            const bool on0 = t < len && p.ok0, on1 = t < len && p.ok1;
            const float4 w = make_float4(on0 ? s0 : 0.0f, on0 ? e.x : 0.0f, on1 ? s1 : 0.0f, on1 ? e.y : 0.0f);
            s_dt[wave][(q * NG + g) * J + j] = w;
            total.x += w.x, total.y += w.z;
        }
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            const int x = e * 64 + lane;
            const bool on = t0 + x / Y::N4 < len && x % Y::N4 < a.n;
            reinterpret_cast<float*>(s_c[wave])[x] = on ? value_of(v.c[e]) : 0.0f;
        }
        if (chunk > first) load_chunk<T, NG, true>(a, p, chunk - 1, v);
        wave_lds_sync();
        const auto walk = [&](auto starts) {
#pragma unroll
        for (int t = SSM_TOK - 1; t >= 0; --t) {
            const float4 x = s_dt[wave][t * J + j], C = s_c[wave][t * NG + g];
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
        }
        };
        if (resets) walk(std::true_type{});
        else walk(std::false_type{});
        wave_lds_sync();
    }
#pragma unroll
    for (int o = 32; o >= J; o >>= 1) {
        total.x += __shfl_xor(total.x, o);
        total.y += __shfl_xor(total.y, o);
    }
    float* at = a.part + (((int64_t)b * a.plan.segments + seg) * 2 * a.n + 4 * g) * a.d + p.c0;
#pragma unroll
    for (int s = 0; s < 4; ++s, at += a.d) {
        if (!okn[s]) continue;
        const float d0 = anew ? 0.0f : __builtin_amdgcn_exp2f(total.x * A[0][s]);
        const float d1 = anew ? 0.0f : __builtin_amdgcn_exp2f(total.y * A[1][s]);
        store_pair(at, make_float2(d0, d1), p.ok0, p.ok1, p.pair);
        store_pair(at + (int64_t)a.n * a.d, make_float2(G[0][s], G[1][s]), p.ok0, p.ok1, p.pair);
    }
}

// Waves of the workgroup hold channels of one group of b and c, side by side.
template <class T, int NG, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void ssm_bwd_kernel(const SsmArgs a) {
    using Y = Lay<NG>;
    constexpr int Q = Y::Q, J = Y::J, N4 = Y::N4, ROW = 68;  // a row of 64 lanes' values, padded
    __shared__ float4 s_dt[WAVES][SSM_TOK * J];               // s, s u of two channels
    __shared__ float2 s_e[WAVES][SSM_TOK * J], s_slope[WAVES][SSM_TOK * J], s_gate[WAVES][SSM_TOK * J];  // e; softplus'; dy (z sigmoid(z))'
    __shared__ float4 s_b[WAVES][SSM_TOK * NG], s_c[WAVES][SSM_TOK * NG];
    __shared__ __align__(16) float s_in[WAVES][8 * ROW];      // a token's values of dc, db by lane
    __shared__ float s_sum[WAVES][SSM_TOK][8 * NG];           // their sums over a wave's channels
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane / J, j = lane % J;
    const int blocks = a.plan.blocks * a.groups, segs = a.plan.segments;
    const int block = blockIdx.x % blocks, seg = blockIdx.x / blocks % segs, b = blockIdx.x / blocks / segs;
    const int gr = block / a.plan.blocks;
    const Place p = place_of<NG>(a, block % a.plan.blocks * WAVES + wave, gr, seg, b);
    const int len = length_of(a, b);

    float A[2][4], G[2][4], dA[2][4];
    bool okn[4];
    load_rates(a, p, g, A, okn);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            G[c][s] = dA[c][s] = 0.0f;
            if (!(c ? p.ok1 : p.ok0) || !okn[s]) continue;
            const int n = 4 * g + s;
            if (a.dh) G[c][s] = a.dh[((int64_t)b * a.d + p.c0 + c) * a.n + n];
            // the cotangent that the segments behind this one hand on
            const float* at = a.part + ((int64_t)b * segs + segs - 1) * 2 * a.n * a.d + (int64_t)n * a.d + p.c0 + c;
            for (int i = segs - 1; i > seg; --i, at -= (int64_t)2 * a.n * a.d) {
                const float decay = at[0], left = at[(int64_t)a.n * a.d];
                G[c][s] = decay == 0.0f ? left : fmaf(decay, G[c][s], left);
            }
        }
    const float2 bias = a.dt_bias ? make_float2(a.dt_bias[p.i], a.dt_bias[p.k]) : make_float2(0.f, 0.f);
    const float2 skip = a.skip ? make_float2(a.skip[p.i], a.skip[p.k]) : make_float2(0.f, 0.f);
    float2 dskip = make_float2(0.f, 0.f), dbias = make_float2(0.f, 0.f);
    const int first = seg * a.plan.seg, last = min(first + a.plan.seg, a.plan.chunks);
    Chunk<T, NG> v;
    if (first < last) load_chunk<T, NG, false>(a, p, last - 1, v);
    for (int chunk = last - 1; chunk >= first; --chunk) {
        const int t0 = chunk * SSM_TOK;
        const uint32_t resets = resets_of(a, b, t0, len);
        float2 us[Q];
        float hin[2][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) hin[0][s] = p.ok0 && okn[s] ? v.h[s].x : 0.0f, hin[1][s] = p.ok1 && okn[s] ? v.h[s].y : 0.0f;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int t = t0 + q * NG + g, at = (q * NG + g) * J + j;
            const bool on0 = t < len && p.ok0, on1 = t < len && p.ok1;
            const float2 x = v.dt[q].get(), dy = v.dy[q].get();
            float2 u = v.u[q].get(), e = dy, slope = make_float2(1.f, 1.f), s = make_float2(x.x + bias.x, x.y + bias.y);
            if (a.softplus) s.x = softplus_of(s.x, &slope.x), s.y = softplus_of(s.y, &slope.y);
            if (a.z) {
                const float2 z = v.z[q].get();
                const float g0 = sigmoid_of(z.x), g1 = sigmoid_of(z.y);
                e.x *= z.x * g0, e.y *= z.y * g1;
                s_gate[wave][at] = make_float2(dy.x * (g0 * (1.0f + z.x * (1.0f - g0))), dy.y * (g1 * (1.0f + z.y * (1.0f - g1))));
            }
            u.x = on0 ? u.x : 0.0f, u.y = on1 ? u.y : 0.0f;  // padding may hold anything
            us[q] = u;
            s_dt[wave][at] = make_float4(on0 ? s.x : 0.0f, on0 ? s.x * u.x : 0.0f, on1 ? s.y : 0.0f, on1 ? s.y * u.y : 0.0f);
            s_e[wave][at] = make_float2(on0 ? e.x : 0.0f, on1 ? e.y : 0.0f);
            s_slope[wave][at] = slope;
        }
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            const int x = e * 64 + lane;
            const bool on = t0 + x / N4 < len && x % N4 < a.n;
            reinterpret_cast<float*>(s_b[wave])[x] = on ? value_of(v.b[e]) : 0.0f;
            reinterpret_cast<float*>(s_c[wave])[x] = on ? value_of(v.c[e]) : 0.0f;
        }
        if (chunk > first) load_chunk<T, NG, false>(a, p, chunk - 1, v);
        wave_lds_sync();

        // a chunk without a sequence's start, as most are, runs free of selects
        const auto walk = [&](auto starts) {
        // the chunk's states; where there is a gate their outputs, for its gradient
        float h[SSM_TOK][2][4];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float y0[NG], y1[NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int t = q * NG + i;
                const float4 x = s_dt[wave][t * J + j], B = s_b[wave][t * NG + g];
                const float bs[4] = {B.x, B.y, B.z, B.w};
                const bool start = decltype(starts)::value && (resets >> t & 1u);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float before0 = start ? 0.0f : t ? h[t - 1][0][s] : hin[0][s], before1 = start ? 0.0f : t ? h[t - 1][1][s] : hin[1][s];
                    h[t][0][s] = fmaf(__builtin_amdgcn_exp2f(x.x * A[0][s]), before0, x.y * bs[s]);
                    h[t][1][s] = fmaf(__builtin_amdgcn_exp2f(x.z * A[1][s]), before1, x.w * bs[s]);
                }
                if (a.z) {
                    const float4 C = s_c[wave][t * NG + g];
                    y0[i] = fmaf(C.w, h[t][0][3], fmaf(C.z, h[t][0][2], fmaf(C.y, h[t][0][1], C.x * h[t][0][0])));
                    y1[i] = fmaf(C.w, h[t][1][3], fmaf(C.z, h[t][1][2], fmaf(C.y, h[t][1][1], C.x * h[t][1][0])));
                }
            }
            if (a.z) {
                const int t = t0 + q * NG + g;
                const float r0 = group_sum<NG>(y0), r1 = group_sum<NG>(y1);
                const float2 k = s_gate[wave][(q * NG + g) * J + j];
                const float2 dz = make_float2(t < len ? k.x * fmaf(skip.x, us[q].x, r0) : 0.0f, t < len ? k.y * fmaf(skip.y, us[q].y, r1) : 0.0f);
                if (t < a.length)
                    store_pair(static_cast<T*>(a.dz) + ((int64_t)b * a.length + t) * a.d + p.c0, dz, p.ok0, p.ok1, p.pair);
            }
        }
#pragma unroll
        for (int q = Q - 1; q >= 0; --q) {
            float gb0[NG], gb1[NG], ar0[NG], ar1[NG];
#pragma unroll
            for (int i = NG - 1; i >= 0; --i) {
                const int t = q * NG + i;
                const float4 x = s_dt[wave][t * J + j], B = s_b[wave][t * NG + g], C = s_c[wave][t * NG + g];
                const float2 e = s_e[wave][t * J + j];
                const float bs[4] = {B.x, B.y, B.z, B.w}, cs[4] = {C.x, C.y, C.z, C.w};
                const bool start = decltype(starts)::value && (resets >> t & 1u);
                float* in = s_in[wave] + lane;
                gb0[i] = gb1[i] = ar0[i] = ar1[i] = 0.0f;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float g0 = fmaf(cs[s], e.x, G[0][s]), g1 = fmaf(cs[s], e.y, G[1][s]);
                    in[s * ROW] = fmaf(e.x, h[t][0][s], e.y * h[t][1][s]);
                    in[(4 + s) * ROW] = fmaf(x.y, g0, x.w * g1);
                    gb0[i] = fmaf(g0, bs[s], gb0[i]), gb1[i] = fmaf(g1, bs[s], gb1[i]);
                    const float w0 = start ? 0.0f : __builtin_amdgcn_exp2f(x.x * A[0][s]) * g0;
                    const float w1 = start ? 0.0f : __builtin_amdgcn_exp2f(x.z * A[1][s]) * g1;
                    const float r0 = start ? 0.0f : w0 * (t ? h[t - 1][0][s] : hin[0][s]), r1 = start ? 0.0f : w1 * (t ? h[t - 1][1][s] : hin[1][s]);
                    ar0[i] = fmaf(r0, A[0][s], ar0[i]), ar1[i] = fmaf(r1, A[1][s], ar1[i]);
                    dA[0][s] = fmaf(x.x, r0, dA[0][s]), dA[1][s] = fmaf(x.z, r1, dA[1][s]);
                    G[0][s] = w0, G[1][s] = w1;
                }
                wave_lds_sync();
                // lane r sums value r / 8 of lanes 8 (r % 8) and the seven behind it
                const float4* from = reinterpret_cast<const float4*>(s_in[wave] + (lane >> 3) * ROW + (lane & 7) * 8);
                const float4 lo = from[0], hi = from[1];
                float* to = s_sum[wave][t] + (lane >> 3) * NG;
                const float l = (lo.x + lo.y) + (lo.z + lo.w), u = (hi.x + hi.y) + (hi.z + hi.w);
                if constexpr (NG == 16) {
                    to[2 * (lane & 7)] = l, to[2 * (lane & 7) + 1] = u;
                } else {
                    float w = l + u;
#pragma unroll
                    for (int o = 1; o < 8 / NG; o <<= 1) w += __shfl_xor(w, o);
                    if ((lane & 7) % (8 / NG) == 0) to[(lane & 7) * NG / 8] = w;
                }
                wave_lds_sync();
            }
            const int t = t0 + q * NG + g, at = (q * NG + g) * J + j;
            const float sb0 = group_sum<NG>(gb0), sb1 = group_sum<NG>(gb1);
            const float sa0 = LN2 * group_sum<NG>(ar0), sa1 = LN2 * group_sum<NG>(ar1);  // A holds a log2 e
            const float4 x = s_dt[wave][at];
            const float2 e = s_e[wave][at], slope = s_slope[wave][at], u = us[q];
            const bool on = t < len;
            const float2 du = make_float2(on ? fmaf(x.x, sb0, skip.x * e.x) : 0.0f, on ? fmaf(x.z, sb1, skip.y * e.y) : 0.0f);
            const float2 dd = make_float2(on ? fmaf(u.x, sb0, sa0) * slope.x : 0.0f, on ? fmaf(u.y, sb1, sa1) * slope.y : 0.0f);
            dskip.x = fmaf(e.x, u.x, dskip.x), dskip.y = fmaf(e.y, u.y, dskip.y);
            dbias.x += dd.x, dbias.y += dd.y;
            if (t < a.length) {
                const int64_t row = ((int64_t)b * a.length + t) * a.d + p.c0;
                store_pair(static_cast<T*>(a.du) + row, du, p.ok0, p.ok1, p.pair);
                store_pair(static_cast<T*>(a.ddt) + row, dd, p.ok0, p.ok1, p.pair);
            }
        }
        };
        if (resets) walk(std::true_type{});
        else walk(std::false_type{});
        __syncthreads();
        for (int x = threadIdx.x; x < SSM_TOK * 8 * NG; x += 64 * WAVES) {
            const int n = x % N4, k = x / N4 % 2, t = x / (2 * N4), at = (k * 4 + n % 4) * NG + n / 4;
            float w = s_sum[0][t][at];
#pragma unroll
            for (int i = 1; i < WAVES; ++i) w += s_sum[i][t][at];
            if (t0 + t < a.length) a.part_bc[(((int64_t)block * a.batch + b) * a.length + t0 + t) * 2 * N4 + k * N4 + n] = w;
        }
        __syncthreads();
    }
    if (seg == 0 && a.dh0) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if ((c ? p.ok1 : p.ok0) && okn[s]) a.dh0[((int64_t)b * a.d + p.c0 + c) * a.n + 4 * g + s] = G[c][s];
    }
    const int64_t mine = (int64_t)b * segs + seg;
    float* at = a.part_a + (mine * a.n + 4 * g) * a.d + p.c0;
#pragma unroll
    for (int s = 0; s < 4; ++s, at += a.d)
        if (okn[s]) store_pair(at, make_float2(dA[0][s], dA[1][s]), p.ok0, p.ok1, p.pair);
#pragma unroll
    for (int o = 32; o >= J; o >>= 1) {
        dskip.x += __shfl_xor(dskip.x, o), dskip.y += __shfl_xor(dskip.y, o);
        dbias.x += __shfl_xor(dbias.x, o), dbias.y += __shfl_xor(dbias.y, o);
    }
    if (g == 0) {
        float* pd = a.part_d + mine * 2 * a.d + p.c0;
        store_pair(pd, dskip, p.ok0, p.ok1, p.pair);
        store_pair(pd + a.d, dbias, p.ok0, p.ok1, p.pair);
    }
}

// Sums of the workgroups' parts, in a fixed order: db and dc over the channels' workgroups (FP32, as they are few), da, dskip
// and ddt_bias over rows and segments (FP64).  The first `bc` workgroups take db and dc.
template <class T>
__global__ __launch_bounds__(256) void ssm_join_kernel(const SsmArgs a, unsigned bc) {
    const int n4 = SSM_STATES * a.plan.ng;
    if (blockIdx.x < bc) {
        const int64_t rows = (int64_t)a.batch * a.length, x = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (x >= rows * a.groups * 2 * n4) return;
        const int n = (int)(x % n4), k = (int)(x / n4 % 2), gr = (int)(x / (2 * n4) / rows);
        const int64_t row = x / (2 * n4) % rows;
        if (n >= a.n) return;
        const float* at = a.part_bc + ((int64_t)gr * a.plan.blocks * rows + row) * 2 * n4 + k * n4 + n;
        float w = 0.0f;
        for (int i = 0; i < a.plan.blocks; ++i) w += at[(int64_t)i * rows * 2 * n4];
        store_value(static_cast<T*>(k ? a.db : a.dc) + (row * a.groups + gr) * a.n + n, w);
        return;
    }
    const int64_t x = (int64_t)(blockIdx.x - bc) * 256 + threadIdx.x;
    const int i = (int)(x % a.d), n = (int)(x / a.d), parts = a.batch * a.plan.segments;
    if (n >= a.n + 2) return;
    const bool rate = n < a.n;
    const float* at = rate ? a.part_a + (int64_t)n * a.d + i : a.part_d + (int64_t)(n - a.n) * a.d + i;
    const int64_t step = rate ? (int64_t)a.n * a.d : 2 * (int64_t)a.d;
    double w = 0.0;
    for (int k = 0; k < parts; ++k) w += (double)at[k * step];
    float* out = rate ? a.da + (int64_t)i * a.n + n : n == a.n ? (a.dskip ? a.dskip + i : nullptr) : (a.ddt_bias ? a.ddt_bias + i : nullptr);
    if (out) *out = (float)w;
}

template <class T, int NG>
void launch_bwd(const SsmArgs& a, hipStream_t s) {
    constexpr int WAVES = NG == 1 ? 2 : 4;
    if (a.plan.segments > 1)
        LRS_LAUNCH(K_SSM_REV, (ssm_rev_kernel<T, NG>),
                   dim3((unsigned)ceil_div((int64_t)a.plan.tiles * a.groups * a.batch * (a.plan.segments - 1), 4)), dim3(256), 0, s, a);
    LRS_LAUNCH(K_SSM_BWD, (ssm_bwd_kernel<T, NG, WAVES>), dim3((unsigned)((int64_t)a.plan.blocks * a.groups * a.plan.segments * a.batch)),
               dim3(64 * WAVES), 0, s, a);
}
template <class T>
void launch_bwd_any(const SsmArgs& a, hipStream_t s) {
    if (a.batch > 0) {
        switch (a.plan.ng) {
            case 1: launch_bwd<T, 1>(a, s); break;
            case 2: launch_bwd<T, 2>(a, s); break;
            case 4: launch_bwd<T, 4>(a, s); break;
            case 8: launch_bwd<T, 8>(a, s); break;
            default: launch_bwd<T, 16>(a, s);
        }
    }
    const unsigned bc = (unsigned)ceil_div((int64_t)a.batch * a.length * a.groups * 2 * SSM_STATES * a.plan.ng, 256);
    LRS_LAUNCH(K_SSM_JOIN, (ssm_join_kernel<T>), dim3(bc + (unsigned)ceil_div((int64_t)a.d * (a.n + 2), 256)), dim3(256), 0, s, a, bc);
}

}  // namespace

hipError_t launch_ssm_bwd(const SsmArgs& a, bool f32, hipStream_t s) {
    if (f32) launch_bwd_any<float>(a, s);
    else launch_bwd_any<uint16_t>(a, s);
    return hipGetLastError();
}

}  // namespace lrs
