// ssm.hpp -- declarations and device helpers of the selective scan and the
// short causal convolution.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "internal.hpp"
#include "ssm_plan.hpp"

namespace lrs {

// ------------------------------------------------------- selective scan ---
struct SsmArgs {
    int batch, length, d, n, groups, per;  // per: channels of a group
    int softplus;
    SsmPlan plan;
    const void *u, *dt, *b, *c, *z;        // rows at a distance
    int64_t u_stride, dt_stride, b_stride, c_stride, z_stride;
    const float *a, *skip, *dt_bias, *h0;
    const uint8_t* reset;
    const int32_t* lengths;
    void* y;
    float *h, *saved;                      // h: final states; saved [batch, chunks, n, d]: the states before each chunk
    float* part;                           // [batch, segments, 2, n, d]: root of the product of a segment's decays (SEGMENT_STARTS: a sequence
                                           // starts in it), state (cotangent) leaving it from zero
    // backward
    const void* dy;
    int64_t dy_stride;
    const float* dh;
    void *du, *ddt, *db, *dc, *dz;
    float *da, *dskip, *ddt_bias, *dh0;
    float* part_bc;                        // [groups * blocks, batch * length, 2, 4 ng]: db, dc of a workgroup's channels
    float* part_a;                         // [batch * segments, n, d]
    float* part_d;                         // [batch * segments, 2, d]: dskip, ddt_bias
};
hipError_t launch_ssm_fwd(const SsmArgs& a, bool f32, hipStream_t s);
hipError_t launch_ssm_bwd(const SsmArgs& a, bool f32, hipStream_t s);
hipError_t launch_ssm_step(const SsmArgs& a, bool f32, hipStream_t s);

// ---------------------------------------------------- causal convolution ---
struct ConvArgs {
    int batch, length, d, width, act;
    int tokens, pieces;                    // tokens of a piece of a row, pieces of a row
    const void* x;
    int64_t x_stride;
    const float *w, *bias;
    const void* state;
    const uint8_t* reset;
    const int32_t* lengths;
    void *y, *state_out;
    // backward
    const void* dy;
    int64_t dy_stride;
    const void* dstate_out;
    void *dx, *dstate;
    float *dw, *dbias;
    float* part;                           // [batch * pieces, width + 1, d]: dw, dbias
};
hipError_t launch_conv_fwd(const ConvArgs& a, bool f32, hipStream_t s);
hipError_t launch_conv_bwd(const ConvArgs& a, bool f32, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs& a, bool f32, hipStream_t s);

// ----------------------------------------------------------- activations ---
constexpr float LOG2E = 1.44269504f, LOG2E_LO = 1.92596303e-8f, LN2 = 0.693147181f;  // LOG2E + LOG2E_LO = log2 e to 48 bits

__device__ __forceinline__ float sigmoid_of(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * x));
}

// log(1 + e^x) and its derivative.  e^x is 2^t with the rounding of t put back; log(1 + e) is taken of the rounded
// 1 + e and scaled by e over what that sum holds of it, so that it keeps FP32's relative precision where e is small
// (D. Goldberg, "What every computer scientist should know about floating-point arithmetic", theorem 4).  Below -110, where e^x is
// less than FP32 holds, x counts as -110: a token masked by the lowest value or minus infinity has s = 0.
__device__ __forceinline__ float softplus_of(float x, float* slope) {
    x = x < -110.0f ? -110.0f : x;
    const float t = x * LOG2E, rest = fmaf(x, LOG2E, -t) + x * LOG2E_LO;
    float e = __builtin_amdgcn_exp2f(t);
    e = fmaf(e * LN2, rest, e);
    const float s = 1.0f + e, part = s - 1.0f;
    const float l = part > 0.0f ? LN2 * __builtin_amdgcn_logf(s) * (e * __builtin_amdgcn_rcpf(part)) : e;
    const bool large = x > 20.0f;  // log(1 + e^-x) is below x's rounding
    *slope = large ? 1.0f : e * __builtin_amdgcn_rcpf(s);
    return large ? x : l;
}

// --------------------------------------------------- pairs of channels ---
typedef f32x2_t __attribute__((aligned(4))) f32x2_a4;
typedef uint32_t __attribute__((aligned(2))) u32_a2;

// Two channels of a row as they lie in memory, at a uniform base and a lane's offset in bytes.
template <class T>
struct Pair;
template <>
struct Pair<uint16_t> {
    uint32_t w;
    static __device__ __forceinline__ Pair load(const char* base, uint32_t off) { return {*reinterpret_cast<const u32_a2*>(base + off)}; }
    static __device__ __forceinline__ Pair one(const uint16_t* p) { return {(uint32_t)*p << 16}; }  // as the second
    static __device__ __forceinline__ Pair load(const char* base, uint32_t off, bool single) {
        return single ? one(reinterpret_cast<const uint16_t*>(base + off)) : load(base, off);
    }
    __device__ __forceinline__ float2 get() const { return make_float2(bf16_lo(w), bf16_hi(w)); }
};
template <>
struct Pair<float> {
    f32x2_t w;
    static __device__ __forceinline__ Pair load(const char* base, uint32_t off) { return {*reinterpret_cast<const f32x2_a4*>(base + off)}; }
    static __device__ __forceinline__ Pair one(const float* p) { return {f32x2_t{0.0f, *p}}; }
    static __device__ __forceinline__ Pair load(const char* base, uint32_t off, bool single) {
        return single ? one(reinterpret_cast<const float*>(base + off)) : load(base, off);
    }
    __device__ __forceinline__ float2 get() const { return make_float2(w[0], w[1]); }
};

__device__ __forceinline__ float value_of(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float value_of(float v) { return v; }
__device__ __forceinline__ void store_value(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_value(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, v); }

// Stores a pair, or the first of it where it has no partner.
template <class T>
__device__ __forceinline__ void store_pair(char* base, uint32_t off, float2 v, bool ok0, bool ok1) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t w = pack_bf16x2(v.x, v.y);
        if (ok1) __builtin_nontemporal_store(w, reinterpret_cast<u32_a2*>(base + off));
        else if (ok0) *reinterpret_cast<uint16_t*>(base + off) = (uint16_t)w;
    } else {
        if (ok1) __builtin_nontemporal_store(f32x2_t{v.x, v.y}, reinterpret_cast<f32x2_a4*>(base + off));
        else if (ok0) *reinterpret_cast<float*>(base + off) = v.x;
    }
}

// ------------------------------------------------- sums over lane groups ---
// The value of the lane whose number differs in bit M.
template <int M>
__device__ __forceinline__ float row_xor(float v) {
    constexpr int ctrl = M == 1 ? 0xb1 : M == 2 ? 0x4e : 0x128;  // quad [1,0,3,2], [2,3,0,1]; rotation of 16 by 8
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), ctrl, 0xf, 0xf, true));
}

// Two values to one: lanes with bit M of their number clear get the sum of a over their pair of lanes, the others that of b.
template <int M>
__device__ __forceinline__ float pair_sum(float a, float b) {
    if constexpr (M == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else if constexpr (M == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else {
        const bool up = threadIdx.x & M;
        if constexpr (M == 8) return (up ? b : a) + row_xor<8>(up ? a : b);
        return (up ? b : a) + __shfl_xor(up ? a : b, M);
    }
}

// v[i] of each of NG tokens to the sum over the NG lane groups: group g gets token g's.
template <int NG>
__device__ __forceinline__ float group_sum(const float (&v)[NG]) {
    float w[NG / 2];
    // the groups' highest bit chooses between the tokens' halves
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) w[i] = pair_sum<32>(v[i], v[i + NG / 2]);
    if constexpr (NG == 2) {
        return w[0];
    } else {
        float x[NG / 4];
#pragma unroll
        for (int i = 0; i < NG / 4; ++i) x[i] = pair_sum<16>(w[i], w[i + NG / 4]);
        if constexpr (NG == 4) return x[0];
        if constexpr (NG == 8) return pair_sum<8>(x[0], x[1]);
        if constexpr (NG == 16) return pair_sum<4>(pair_sum<8>(x[0], x[2]), pair_sum<8>(x[1], x[3]));
    }
}

}  // namespace lrs
