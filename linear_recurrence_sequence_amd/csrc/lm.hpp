// lm.hpp -- declarations and device helpers shared by the language-model
// operators (block norms, linear cross entropy, AdamW, embedding lookup).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "internal.hpp"

namespace lrs {

// ------------------------------------------------- element-aligned loads ---
// Rows of odd width and views into flat buffers are aligned to their element
// type only.  The vector types below say so; gfx950 takes such addresses in
// the same 8- and 16-byte instructions.
typedef u32x2_t __attribute__((aligned(2))) u32x2_a2;
typedef u32x4_t __attribute__((aligned(2))) u32x4_a2;
typedef f32x4_t __attribute__((aligned(4))) f32x4_a4;
typedef uint32_t __attribute__((aligned(1))) u32_a1;

// Four consecutive elements as they lie in memory, for BF16 (T = uint16_t) or FP32.
template <class T>
struct Quad;

template <>
struct Quad<uint16_t> {
    u32x2_t w;
    static __device__ __forceinline__ Quad load(const uint16_t* p) {
        return {__builtin_nontemporal_load(reinterpret_cast<const u32x2_a2*>(p))};
    }
    static __device__ __forceinline__ Quad load_some(const uint16_t* p, int n) {  // the first n < 4, zeros behind
        const uint32_t a = n > 0 ? p[0] : 0u, b = n > 1 ? p[1] : 0u, c = n > 2 ? p[2] : 0u;
        return {u32x2_t{a | b << 16, c}};
    }
    static __device__ __forceinline__ Quad zero() { return {u32x2_t{0u, 0u}}; }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = bf16_lo(w[0]);
        f[1] = bf16_hi(w[0]);
        f[2] = bf16_lo(w[1]);
        f[3] = bf16_hi(w[1]);
    }
    static __device__ __forceinline__ void store(uint16_t* p, const float* f) {
        __builtin_nontemporal_store(u32x2_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])},
                                    reinterpret_cast<u32x2_a2*>(p));
    }
    static __device__ __forceinline__ void store_some(uint16_t* p, const float* f, int n) {
        const uint32_t a = pack_bf16x2(f[0], f[1]), b = pack_bf16x2(f[2], f[3]);
        if (n > 0) p[0] = (uint16_t)a;
        if (n > 1) p[1] = (uint16_t)(a >> 16);
        if (n > 2) p[2] = (uint16_t)b;
    }
};

template <>
struct Quad<float> {
    f32x4_t w;
    static __device__ __forceinline__ Quad load(const float* p) {
        return {__builtin_nontemporal_load(reinterpret_cast<const f32x4_a4*>(p))};
    }
    static __device__ __forceinline__ Quad load_some(const float* p, int n) {
        return {f32x4_t{n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, 0.f}};
    }
    static __device__ __forceinline__ Quad zero() { return {f32x4_t{0.f, 0.f, 0.f, 0.f}}; }
    __device__ __forceinline__ void get(float* f) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = w[i];
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        __builtin_nontemporal_store(f32x4_t{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4_a4*>(p));
    }
    static __device__ __forceinline__ void store_some(float* p, const float* f, int n) {
        if (n > 0) p[0] = f[0];
        if (n > 1) p[1] = f[1];
        if (n > 2) p[2] = f[2];
    }
};

// Rows in groups of four elements.  Where
// the width is no multiple of 4 (TAIL) the group that the row ends in is loaded as the
// row's last four elements and put in place by take(), so that no load stands in a
// branch of its own (each would be waited for there).
template <class T, bool TAIL>
__device__ __forceinline__ Quad<T> row_load(const T* row, int col, int d) {
    if (TAIL) {
        if (d < 4) return col < d ? Quad<T>::load_some(row, d) : Quad<T>::zero();
        return Quad<T>::load(row + (col + 4 <= d ? col : d - 4));
    }
    if (col + 4 <= d) return Quad<T>::load(row + col);
    return Quad<T>::zero();
}
template <bool TAIL, class T>
__device__ __forceinline__ void take(const Quad<T>& q, int col, int d, float* f) {
    q.get(f);
    if (TAIL) {
        const int n = d < 4 && col < d ? 4 : d - col;  // this lane's elements, 4 or more: all
        if (n < 4) {
            const float a = f[1], b = f[2], c = f[3];
            f[0] = n == 3 ? a : n == 2 ? b : n == 1 ? c : 0.0f;
            f[1] = n == 3 ? b : n == 2 ? c : 0.0f;
            f[2] = n == 3 ? c : 0.0f;
            f[3] = 0.0f;
        }
    }
}
template <class T, bool TAIL>
__device__ __forceinline__ void row_store(T* row, int col, int d, const float* f) {
    if (col + 4 <= d) Quad<T>::store(row + col, f);
    else if (TAIL && col < d) Quad<T>::store_some(row + col, f, d - col);
}

// ---------------------------------------------------------- block norms ---
struct NormArgs {
    int64_t rows;
    int d, gate_act;
    float eps;
    const void *x, *y, *gate;
    int64_t x_stride, y_stride, gate_stride;
    const float *w_post, *scale, *w_pre;
    // forward
    void *r, *n;
    float* stats;
    // backward
    const void *dr, *dn;
    int64_t dr_stride, dn_stride;
    void *dx, *dy, *dgate;
    float* part;  // [blocks, 2, d]: sum dn rh, sum v act yh
};
int lm_norm_bwd_blocks(int64_t rows, int d);
hipError_t launch_norm_fwd(const NormArgs& a, int stream_f32, int branch_f32, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, int stream_f32, int branch_f32, float* dw_post, float* dscale,
                           float* dw_pre, hipStream_t s);

// ---------------------------------------------------------------- AdamW ---
constexpr int ADAMW_LAUNCH = 48;     // tensors a launch takes (its arguments hold them)
constexpr int ADAMW_CHUNK = 4096;    // elements a workgroup updates
struct AdamwArgs {
    int count;
    float b1, c1, b2, c2, step_size, root_scale, eps;  // c = 1 - b; step_size = lr / (1 - b1^t); root_scale = (1 - b2^t)^-1/2
    uint32_t start[ADAMW_LAUNCH];    // first workgroup of each tensor
    float decay[ADAMW_LAUNCH];       // lr decay
    int64_t n[ADAMW_LAUNCH];
    void* p[ADAMW_LAUNCH];
    const void* g[ADAMW_LAUNCH];
    void *m[ADAMW_LAUNCH], *v[ADAMW_LAUNCH];
    float *master[ADAMW_LAUNCH], *m_scale[ADAMW_LAUNCH], *v_scale[ADAMW_LAUNCH];
};
hipError_t launch_adamw(const AdamwArgs& a, uint32_t blocks, int param_f32, int grad_f32, bool master, bool bits8,
                        hipStream_t s);

// -------------------------------------------------- linear cross entropy ---
struct CeToken {    // a token as the backward takes it
    float c, base, dl;  // (dloss + dlse) / scale, lse in base 2, dloss / scale
    int target;         // -1: none
};
struct CeArgs {
    int n, d, v;                // tokens, width, vocabulary
    float cap;                  // 0: logits are not capped
    const void* h;              // bf16 [n, d], row stride h_stride
    int64_t h_stride;
    const void* w;              // bf16 [v, d]
    const int64_t* target;      // [n]; negative: the token does not count
    // forward
    float* part;                // [ce_parts(n, d, v), n] (maximum, sum of 2^(z - maximum)), base-2 logits
    float* picked;              // [n] logit of the target
    float *loss, *lse;          // [n]
    // backward
    const float *lse_in, *dloss, *dlse;
    float* scale;               // [1] what dz is divided by
    int* active;                // [1] tokens that take part
    int *list, *place;          // [n] their numbers; place in the list, -1 of the others
    CeToken* token;             // [active]
    void* packed;               // bf16 [active, d] their rows of h
    void* dz;                   // bf16 [active, chunk], or [chunk, few]
    float* dh_part;             // [splits, n, d], rows as listed
    void *dh, *dw;
    int grad_f32;
    int few;                    // columns of dz laid out [chunk, few]; 0: [active, chunk]
};
hipError_t launch_ce_fwd(const CeArgs& a, hipStream_t s);
hipError_t launch_ce_bwd(const CeArgs& a, hipStream_t s);

// ------------------------------------------------------ embedding lookup ---
constexpr int EMBED_ROWS = 512;   // rows of the vocabulary that a sorting workgroup takes
constexpr int EMBED_WAVES = 16;   // of a sorting workgroup
// The sort is the launch with the most threads for a row, two, in whole workgroups.
constexpr int64_t EMBED_MOST_V = MOST_THREADS / (64 * EMBED_WAVES) * EMBED_ROWS;
constexpr int EMBED_RUN = 32;     // tokens that one wave adds up for a row
struct EmbedArgs {
    int64_t n, v;                 // tokens, rows of the vocabulary
    int d;
    float scale;
    const int64_t* tokens;        // [n]; negative: padding
    const void* w;                // [v, d]
    void* out;                    // [n, d]
    // backward
    const void* dout;             // [n, d], row stride dout_stride
    int64_t dout_stride;
    void* dw;                     // [v, d]
    int add;                      // to what dw holds
    int *start, *order;           // [v + 1], [n]: where each row's tokens begin in the order
    float* part;                  // [ceil(n / EMBED_RUN), 2, d]: what a run holds of the row that it begins and ends in
};
hipError_t launch_embed_fwd(const EmbedArgs& a, bool w_f32, bool out_f32, hipStream_t s);
hipError_t launch_embed_bwd(const EmbedArgs& a, bool out_f32, bool grad_f32, hipStream_t s);

}  // namespace lrs
