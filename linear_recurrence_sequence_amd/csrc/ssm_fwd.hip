// ssm_fwd.hip -- the selective state space scan, forward, and its step for
// single tokens.
//
// For every channel i and state j (x_t = dt_t + dt_bias, s_t = softplus(x_t)):
//   h_t = exp(s_t a) h_{t-1} + s_t u_t b_t,  y_t = (sum_j c_t h_t + d u_t) z_t sigmoid(z_t).
//
// Bound by the vector ALU: each state of each token takes an exponential (two issue slots), two products and two
// multiply-adds, and as decays differ by channel and state no matrix product can do it.  So states stay in registers, and
// what one value serves many lanes is formed once: s and s u for a chunk of 16 tokens by the lanes that hold a token each,
// through LDS to the lanes that hold the states.  A wave holds two channels by four states a lane: of 16 states its lanes are four
// groups of states of 16 channel pairs, so that a value from LDS serves four or eight states and the sum over states is
// in the lane but for two steps, which are taken for four tokens at once.
//
// 32768 x 2048 channels x 16 states in BF16, gated and packed: the segments from zero 240 us, the scan with the states kept for
// the backward 350 us, 3.0 T state updates a second; the vector ALU is busy for 81 and 79% of the time.
// Registers of the gated scan, and waves a SIMD (BF16; FP32): up to 8 states 154, three (169, two); 9 to 16 138, three (150, three);
// 17 to 32 181, two (187, two); 33 to 64 288, one (291, one), as a token's sums over 16 lane groups are formed for 16 tokens at once.  Nothing spills.
#include "ssm_lay.hpp"

namespace lrs {
namespace {

// A chunk's values as they lie in memory.
template <class T, int NG>
struct Chunk {
    static constexpr int Q = Lay<NG>::Q;
    Pair<T> u[Q], dt[Q], z[Q];
    T b[NG], c[NG];
};
template <class T, int NG, bool GATE, bool SUM>
__device__ __forceinline__ void load_chunk(const SsmArgs& a, const Place& p, int chunk, Chunk<T, NG>& v) {
    const int64_t row0 = (int64_t)p.b * a.length + chunk * SSM_TOK;
    const int left = a.length - chunk * SSM_TOK, g = fresh_lane() / Lay<NG>::J;
    const char *u = rows_at<T>(a.u, row0, a.u_stride), *dt = rows_at<T>(a.dt, row0, a.dt_stride), *z = rows_at<T>(a.z, row0, a.z_stride);
    both_ways(a.per == 1, [&](auto single) {
#pragma unroll
        for (int q = 0; q < Lay<NG>::Q; ++q) {
            const int r = min(q * NG + g, left - 1);
            v.u[q] = Pair<T>::load(u, row_off<T>(r, a.u_stride, p.i), decltype(single)::value);
            v.dt[q] = Pair<T>::load(dt, row_off<T>(r, a.dt_stride, p.i), decltype(single)::value);
            if (!SUM && GATE) v.z[q] = Pair<T>::load(z, row_off<T>(r, a.z_stride, p.i), decltype(single)::value);
        }
    });
    load_group<T, NG>(a.b, a.b_stride, row0, left, p.gr, a.n, v.b);
    if (!SUM) load_group<T, NG>(a.c, a.c_stride, row0, left, p.gr, a.n, v.c);
}

// SUM: a segment from a zero state, for the product of its decays and the state that leaves it.
template <class T, int NG, bool GATE, bool SUM>
__global__ __launch_bounds__(256) void ssm_fwd_kernel(const SsmArgs a) {
    using Y = Lay<NG>;
    constexpr int Q = Y::Q, J = Y::J;
    struct Wave {
        float4 su[SSM_TOK * J];                        // s, s u of two channels
        float4 b[SSM_TOK * NG], c[SUM ? 1 : SSM_TOK * NG];
    };
    __shared__ Wave waves[4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = a.plan.tiles * a.groups, segs = SUM ? a.plan.segments - 1 : a.plan.segments;
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit >= (int64_t)tiles * segs * a.batch) return;  // waves do not wait for each other
    const int tile = (int)(unit % tiles), seg = (int)(unit / tiles % segs), b = (int)(unit / tiles / segs);
    const Place p = place_of<NG>(a, tile % a.plan.tiles, tile / a.plan.tiles, seg, b);
    const int len = length_of(a, b);
    Wave& m = waves[wave];

    float A[2][4], h[2][4];
    bool okn[4];
    load_rates(a, p, A, okn);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            h[c][s] = 0.0f;
            if (SUM || !(c ? p.ok1 : p.ok0) || !okn[s]) continue;
            const int n = 4 * p.g + s;
            if (a.h0) h[c][s] = a.h0[((int64_t)b * a.d + p.c0 + c) * a.n + n];
        }
    if (!SUM) through_segments(a, p, 0, seg, 1, h);  // what those before this one leave
#pragma unroll
    for (int s = 0; s < 4; ++s) h[0][s] = p.ok0 && okn[s] ? h[0][s] : 0.0f, h[1][s] = p.ok1 && okn[s] ? h[1][s] : 0.0f;
    const float2 bias = load_two(a, a.dt_bias, p), skip = load_two(a, SUM ? nullptr : a.skip, p);
    float2 total = make_float2(0.f, 0.f);
    bool anew = false;
    const int first = seg * a.plan.seg, last = min(first + a.plan.seg, a.plan.chunks);
    Chunk<T, NG> v;
    if (first < last) load_chunk<T, NG, GATE, SUM>(a, p, first, v);
    for (int chunk = first; chunk < last; ++chunk) {
        const uint32_t lane = fresh_lane();
        const int g = lane / J, j = lane % J;
        const int t0 = chunk * SSM_TOK, live = len - t0, left = a.length - t0;
        if (!SUM && a.saved) {
            char* at = reinterpret_cast<char*>(a.saved + ((int64_t)b * a.plan.chunks + chunk) * a.n * a.d);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (okn[s]) store_pair<float>(at, state_off(a, 4 * g + s, p.c0), make_float2(h[0][s], h[1][s]), p.ok0, p.ok1);
        }
        const uint32_t resets = resets_of(a, b, t0);
        anew |= resets != 0;
        float2 us[Q], gate[Q];
        const auto stage = [&](auto mask, auto soft) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                float2 u = own(v.u[q].get(), p);
                const float2 x = own(v.dt[q].get(), p);
                float slope, s0 = x.x + bias.x, s1 = x.y + bias.y;
                if (decltype(soft)::value) s0 = softplus_of(s0, &slope), s1 = softplus_of(s1, &slope);
                if (decltype(mask)::value) {  // padding may hold anything
                    const bool on = q * NG + g < live;
                    s0 = on ? s0 : 0.0f, s1 = on ? s1 : 0.0f;
                    u.x = on ? u.x : 0.0f, u.y = on ? u.y : 0.0f;
                }
                m.su[q * 64 + lane] = make_float4(s0, s0 * u.x, s1, s1 * u.y);
                if (SUM) {
                    total.x += s0, total.y += s1;
                } else {
                    us[q] = u;
                    gate[q] = make_float2(1.0f, 1.0f);
                    if (GATE) {
                        const float2 z = own(v.z[q].get(), p);
                        gate[q] = make_float2(z.x * sigmoid_of(z.x), z.y * sigmoid_of(z.y));
                    }
                }
            }
            put_group<decltype(mask)::value, T, NG>(v.b, m.b, live, a.n);
            if (!SUM) put_group<decltype(mask)::value, T, NG>(v.c, m.c, live, a.n);
        };
        both_ways(!whole_chunk<NG>(a, p.tile, live), [&](auto mask) { both_ways(a.softplus, [&](auto soft) { stage(mask, soft); }); });
        if (chunk + 1 < last) load_chunk<T, NG, GATE, SUM>(a, p, chunk + 1, v);
        wave_lds_sync();
        // a chunk without a sequence's start, as most are, runs free of branches
        const auto walk = [&](auto starts) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                float y0[NG], y1[NG];
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const int t = q * NG + i;
                    const float4 x = m.su[t * J + j], B = m.b[t * NG + g];
                    if (decltype(starts)::value && (resets >> t & 1u)) {
#pragma unroll
                        for (int s = 0; s < 4; ++s) h[0][s] = h[1][s] = 0.0f;
                    }
                    const float bs[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        h[0][s] = fmaf(__builtin_amdgcn_exp2f(x.x * A[0][s]), h[0][s], x.y * bs[s]);
                        h[1][s] = fmaf(__builtin_amdgcn_exp2f(x.z * A[1][s]), h[1][s], x.w * bs[s]);
                    }
                    if (!SUM) {
                        const float4 C = m.c[t * NG + g];
                        y0[i] = fmaf(C.w, h[0][3], fmaf(C.z, h[0][2], fmaf(C.y, h[0][1], C.x * h[0][0])));
                        y1[i] = fmaf(C.w, h[1][3], fmaf(C.z, h[1][2], fmaf(C.y, h[1][1], C.x * h[1][0])));
                    }
                    if (t % 2) __builtin_amdgcn_sched_barrier(0);  // keeps the reads of later tokens from taking all registers
                }
                if (!SUM) {
                    const int r = q * NG + g;
                    const float r0 = group_sum<NG>(y0), r1 = group_sum<NG>(y1);
                    const bool on = r < live;  // padding: whatever u and z hold
                    const float2 y = make_float2(on ? fmaf(skip.x, us[q].x, r0) * gate[q].x : 0.0f, on ? fmaf(skip.y, us[q].y, r1) * gate[q].y : 0.0f);
                    store_pair<T>(rows_at<T>(a.y, (int64_t)b * a.length + t0, a.d), row_off<T>(r, a.d, p.c0), y, r < left && p.ok0, r < left && p.ok1);
                }
            }
        };
        both_ways(resets != 0, walk);
        wave_lds_sync();
    }
    if (SUM) {
        put_segment<NG>(a, p, A, okn, total, anew, h);
    } else if (seg == segs - 1) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if ((c ? p.ok1 : p.ok0) && okn[s]) a.h[((int64_t)b * a.d + p.c0 + c) * a.n + 4 * p.g + s] = h[c][s];
    }
}

// One token.  Bound by reading and writing the states: a lane holds four consecutive states of one channel, LC lanes a
// channel, so that a wave's loads are whole lines whatever n is.
template <class T, int LC>
__global__ __launch_bounds__(256) void ssm_step_kernel(const SsmArgs a) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, row = at / LC;
    const int q = (int)(at % LC), n0 = 4 * q;
    const bool on = row < (int64_t)a.batch * a.d;
    const int b = on ? (int)(row / a.d) : 0, i = on ? (int)(row % a.d) : 0, gr = i / a.per, here = on ? min(max(a.n - n0, 0), 4) : 0;
    float* hp = a.h + ((int64_t)b * a.d + i) * a.n + n0;
    const float* ap = a.a + (int64_t)i * a.n + n0;
    const T* bp = static_cast<const T*>(a.b) + b * a.b_stride + (int64_t)gr * a.n + n0;
    const T* cp = static_cast<const T*>(a.c) + b * a.c_stride + (int64_t)gr * a.n + n0;
    float h[4], A[4], B[4], C[4];
    typedef f32x4_t __attribute__((aligned(4))) f32x4_e;
    if (here == 4) {
        const f32x4_t x = *reinterpret_cast<const f32x4_e*>(hp), y = *reinterpret_cast<const f32x4_e*>(ap);
#pragma unroll
        for (int s = 0; s < 4; ++s) h[s] = x[s], A[s] = y[s], B[s] = value_of(bp[s]), C[s] = value_of(cp[s]);
    } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bool k = s < here;
            h[s] = k ? hp[s] : 0.0f, A[s] = k ? ap[s] : 0.0f, B[s] = k ? value_of(bp[s]) : 0.0f, C[s] = k ? value_of(cp[s]) : 0.0f;
        }
    }
    const float u = value_of(static_cast<const T*>(a.u)[b * a.u_stride + i]);
    float s = value_of(static_cast<const T*>(a.dt)[b * a.dt_stride + i]) + (a.dt_bias ? a.dt_bias[i] : 0.0f), slope;
    const float z = a.z ? value_of(static_cast<const T*>(a.z)[b * a.z_stride + i]) : 0.0f, skip = a.skip ? a.skip[i] : 0.0f;
    if (a.softplus) s = softplus_of(s, &slope);
    const float su = s * u;
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = fmaf(__builtin_amdgcn_exp2f(s * (LOG2E * A[k])), h[k], su * B[k]);
        y = fmaf(C[k], h[k], y);
    }
    if (here == 4) {
        *reinterpret_cast<f32x4_e*>(hp) = f32x4_t{h[0], h[1], h[2], h[3]};
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < here) hp[k] = h[k];
    }
#pragma unroll
    for (int o = LC / 2; o > 0; o >>= 1) y += __shfl_xor(y, o);
    if (on && q == 0) {
        y = fmaf(skip, u, y);
        if (a.z) y *= z * sigmoid_of(z);
        store_value(static_cast<T*>(a.y) + (int64_t)b * a.d + i, y);
    }
}

template <class T, int NG>
void launch_fwd(const SsmArgs& a, hipStream_t s) {
    const int64_t tiles = (int64_t)a.plan.tiles * a.groups * a.batch;
    const dim3 g((unsigned)ceil_div(tiles * a.plan.segments, 4)), b(256);
    if (a.plan.segments > 1)
        LRS_LAUNCH(K_SSM_SUMMARY, (ssm_fwd_kernel<T, NG, false, true>), dim3((unsigned)ceil_div(tiles * (a.plan.segments - 1), 4)), b, 0, s, a);
    if (a.z) LRS_LAUNCH(K_SSM_SCAN, (ssm_fwd_kernel<T, NG, true, false>), g, b, 0, s, a);
    else LRS_LAUNCH(K_SSM_SCAN, (ssm_fwd_kernel<T, NG, false, false>), g, b, 0, s, a);
}
template <class T>
void launch_fwd_any(const SsmArgs& a, hipStream_t s) {
    switch (a.plan.ng) {
        case 2: return launch_fwd<T, 2>(a, s);
        case 4: return launch_fwd<T, 4>(a, s);
        case 8: return launch_fwd<T, 8>(a, s);
        default: return launch_fwd<T, 16>(a, s);
    }
}
template <class T, int LC>
void launch_step(const SsmArgs& a, hipStream_t s) {
    LRS_LAUNCH(K_SSM_STEP, (ssm_step_kernel<T, LC>), dim3((unsigned)ceil_div((int64_t)a.batch * a.d * LC, 256)), dim3(256), 0, s, a);
}
template <class T>
void launch_step_any(const SsmArgs& a, hipStream_t s) {
    switch (a.plan.ng) {
        case 1: return launch_step<T, 1>(a, s);
        case 2: return launch_step<T, 2>(a, s);
        case 4: return launch_step<T, 4>(a, s);
        case 8: return launch_step<T, 8>(a, s);
        default: return launch_step<T, 16>(a, s);
    }
}

}  // namespace

hipError_t launch_ssm_fwd(const SsmArgs& a, bool f32, hipStream_t s) {
    if (f32) launch_fwd_any<float>(a, s);
    else launch_fwd_any<uint16_t>(a, s);
    return hipGetLastError();
}

hipError_t launch_ssm_step(const SsmArgs& a, bool f32, hipStream_t s) {
    if (f32) launch_step_any<float>(a, s);
    else launch_step_any<uint16_t>(a, s);
    return hipGetLastError();
}

}  // namespace lrs
