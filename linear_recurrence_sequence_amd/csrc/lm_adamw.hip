// lm_adamw.hip -- the AdamW step over many tensors in one launch, with the
// two moments in FP32 or in 8 bits.
//
// For every element (FP32 arithmetic):
//   m' = b1 m + (1-b1) g,  v' = b2 v + (1-b2) g^2,
//   p' = p - (lr decay p + step_size m' / (sqrt(v') root_scale + eps)).
// 8-bit moments: blocks of 256 consecutive elements hold e4m3 codes and one
// FP32 scale, max(|.|) / 448.  The second moment is held as its square root,
// which halves the range its codes have to span; a positive root takes at
// least the least code 2^-9, so that an element whose root is far below its
// block's largest still has a divisor.
//
// Bound by memory: 16 bytes an element with a BF16 weight, an FP32 copy and
// 8-bit moments, 28 with FP32 weights and moments.  A lane holds 4 consecutive
// elements, so a wave's 64 lanes hold exactly one block and its maximum is one
// reduction over the wave; a wave requests 4 blocks before it uses the first.
// 0.42 G weights with a BF16 copy and 8-bit moments take 1175 us, 5.7 TB/s; 58 M with
// 32-bit ones 277 us, 6.0 TB/s (a large copy: 4.7 to 4.9 TB/s).
#include <float.h>

#include "lm.hpp"

namespace lrs {
namespace {

constexpr int U = 4;  // blocks of 256 elements a wave holds at once

// The largest |x| of the wave as FP32 bits: an unsigned maximum of the bits
// without sign orders finite < inf < NaN, so a NaN is kept.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// Scale of one block and the codes of this lane's four values.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode(const float* x, float* scale) {
#pragma clang fp contract(off)
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    const float s = __uint_as_float(wave_umax(top)) * (1.0f / 448.0f);
    *scale = s < 0x1p-96f ? 0x1p-96f : s;
    const float inv = 1.0f / *scale;
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = x[i] * inv;
        if (ROOT && x[i] > 0.0f && q[i] < 0x1p-9f) q[i] = 0x1p-9f;
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    return (uint32_t)w;
}

__device__ __forceinline__ void decode(uint32_t w, float s, float* x) {
    x[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0) * s;
    x[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * s;
    x[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * s;
    x[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * s;
}

// Four code bytes; the first n where fewer belong to the tensor.
__device__ __forceinline__ uint32_t code_some(const uint8_t* p, int n) {
    return (n > 0 ? p[0] : 0u) | (n > 1 ? (uint32_t)p[1] << 8 : 0u) | (n > 2 ? (uint32_t)p[2] << 16 : 0u);
}

// The new moments, each operation rounded by itself and the root correctly
// rounded: a code is chosen at the borders between two values, so that every
// evaluation of the formulas in FP32 has to come to the same codes.
__device__ __forceinline__ void moments(const AdamwArgs& a, float g, float* m, float* v, float* root) {
#pragma clang fp contract(off)
    *m = *m * a.b1 + g * a.c1;
    *v = *v * a.b2 + (g * g) * a.c2;
    *root = sqrtf(*v);
}

template <class PT, class GT, bool MASTER, bool BITS8, bool TAIL>
__device__ __forceinline__ void update(const AdamwArgs& a, int t, int64_t base, int64_t n) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t first = base + (int64_t)wave * (U * 256);
    PT* p = static_cast<PT*>(a.p[t]);
    const GT* g = static_cast<const GT*>(a.g[t]);
    Quad<PT> qp[U];
    Quad<GT> qg[U];
    Quad<float> qw[U], qm[U], qv[U];
    uint32_t cm[U], cv[U];
    float sm[U], sv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = first + u * 256 + lane * 4;
        // a lane's elements: all four, or (at the tensor's end) k < 4 of them
        const int k = TAIL ? (int)(n - e < 0 ? 0 : n - e > 4 ? 4 : n - e) : 4;
        if (!TAIL || k == 4) {
            qg[u] = Quad<GT>::load(g + e);
            if (MASTER) qw[u] = Quad<float>::load(a.master[t] + e);
            else qp[u] = Quad<PT>::load(p + e);
            if (BITS8) {
                cm[u] = *reinterpret_cast<const u32_a1*>(static_cast<const uint8_t*>(a.m[t]) + e);
                cv[u] = *reinterpret_cast<const u32_a1*>(static_cast<const uint8_t*>(a.v[t]) + e);
            } else {
                qm[u] = Quad<float>::load(static_cast<const float*>(a.m[t]) + e);
                qv[u] = Quad<float>::load(static_cast<const float*>(a.v[t]) + e);
            }
        } else {
            qg[u] = Quad<GT>::load_some(g + e, k);
            if (MASTER) qw[u] = Quad<float>::load_some(a.master[t] + e, k);
            else qp[u] = Quad<PT>::load_some(p + e, k);
            if (BITS8) {
                cm[u] = code_some(static_cast<const uint8_t*>(a.m[t]) + e, k);
                cv[u] = code_some(static_cast<const uint8_t*>(a.v[t]) + e, k);
            } else {
                qm[u] = Quad<float>::load_some(static_cast<const float*>(a.m[t]) + e, k);
                qv[u] = Quad<float>::load_some(static_cast<const float*>(a.v[t]) + e, k);
            }
        }
        if (BITS8) {
            const int64_t b = (first >> 8) + u;
            const bool in = !TAIL || (b << 8) < n;
            sm[u] = in ? a.m_scale[t][b] : 0.0f;
            sv[u] = in ? a.v_scale[t][b] : 0.0f;
        }
    }
    const float taken = a.decay[t];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t e = first + u * 256 + lane * 4;
        const int k = TAIL ? (int)(n - e < 0 ? 0 : n - e > 4 ? 4 : n - e) : 4;
        float gg[4], pp[4], m[4], v[4], root[4];
        qg[u].get(gg);
        if (MASTER) qw[u].get(pp);
        else qp[u].get(pp);
        if (BITS8) {
            decode(cm[u], sm[u], m);
            decode(cv[u], sv[u], v);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= v[i];
        } else {
            qm[u].get(m);
            qv[u].get(v);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            moments(a, gg[i], &m[i], &v[i], &root[i]);
            // the reciprocal is the hardware's, within one unit in the last place
            const float upd = m[i] * __builtin_amdgcn_rcpf(root[i] * a.root_scale + a.eps);
            // What is taken is summed first: 1 - lr decay in FP32 would round a small decay to a multiple of 2^-24, the same for every
            // element and step.  An infinite weight stays so.
            pp[i] -= fmaf(a.step_size, upd, taken * __builtin_amdgcn_fmed3f(pp[i], -FLT_MAX, FLT_MAX));
        }
        uint32_t em = 0, ev = 0;
        float ns, nr;
        if (BITS8) {
            em = encode<false>(m, &ns);
            ev = encode<true>(root, &nr);
        }
        if (!TAIL || k == 4) {
            if (MASTER) Quad<float>::store(a.master[t] + e, pp);
            Quad<PT>::store(p + e, pp);
            if (BITS8) {
                *reinterpret_cast<u32_a1*>(static_cast<uint8_t*>(a.m[t]) + e) = em;
                *reinterpret_cast<u32_a1*>(static_cast<uint8_t*>(a.v[t]) + e) = ev;
            } else {
                Quad<float>::store(static_cast<float*>(a.m[t]) + e, m);
                Quad<float>::store(static_cast<float*>(a.v[t]) + e, v);
            }
        } else if (k > 0) {
            if (MASTER) Quad<float>::store_some(a.master[t] + e, pp, k);
            Quad<PT>::store_some(p + e, pp, k);
            if (BITS8) {
                for (int i = 0; i < k; ++i) {
                    static_cast<uint8_t*>(a.m[t])[e + i] = (uint8_t)(em >> 8 * i);
                    static_cast<uint8_t*>(a.v[t])[e + i] = (uint8_t)(ev >> 8 * i);
                }
            } else {
                Quad<float>::store_some(static_cast<float*>(a.m[t]) + e, m, k);
                Quad<float>::store_some(static_cast<float*>(a.v[t]) + e, v, k);
            }
        }
        if (BITS8 && lane == 0) {
            const int64_t b = (first >> 8) + u;
            if (!TAIL || (b << 8) < n) {
                a.m_scale[t][b] = ns;
                a.v_scale[t][b] = nr;
            }
        }
    }
}

template <class PT, class GT, bool MASTER, bool BITS8>
__global__ __launch_bounds__(256) void adamw_kernel(const AdamwArgs a) {
    // the tensor this workgroup belongs to: the last one that starts at or
    // before it (scalar compares; the starts come with the arguments)
    int t = 0;
#pragma unroll
    for (int i = 1; i < ADAMW_LAUNCH; ++i) t += (i < a.count && a.start[i] <= blockIdx.x) ? 1 : 0;
    const int64_t base = (int64_t)(blockIdx.x - a.start[t]) * ADAMW_CHUNK, n = a.n[t];
    if (base + ADAMW_CHUNK <= n) update<PT, GT, MASTER, BITS8, false>(a, t, base, n);
    else update<PT, GT, MASTER, BITS8, true>(a, t, base, n);
}

template <class PT, class GT>
void launch_typed(const AdamwArgs& a, uint32_t blocks, bool master, bool bits8, hipStream_t s) {
    const dim3 g(blocks), b(256);
    if (master) {
        if (bits8) LRS_LAUNCH(K_LM_ADAMW, (adamw_kernel<PT, GT, true, true>), g, b, 0, s, a);
        else LRS_LAUNCH(K_LM_ADAMW, (adamw_kernel<PT, GT, true, false>), g, b, 0, s, a);
    } else {
        if (bits8) LRS_LAUNCH(K_LM_ADAMW, (adamw_kernel<PT, GT, false, true>), g, b, 0, s, a);
        else LRS_LAUNCH(K_LM_ADAMW, (adamw_kernel<PT, GT, false, false>), g, b, 0, s, a);
    }
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, uint32_t blocks, int param_f32, int grad_f32, bool master, bool bits8,
                        hipStream_t s) {
    if (param_f32) {
        if (grad_f32) launch_typed<float, float>(a, blocks, master, bits8, s);
        else launch_typed<float, uint16_t>(a, blocks, master, bits8, s);
    } else {
        if (grad_f32) launch_typed<uint16_t, float>(a, blocks, master, bits8, s);
        else launch_typed<uint16_t, uint16_t>(a, blocks, master, bits8, s);
    }
    return hipGetLastError();
}

}  // namespace lrs
