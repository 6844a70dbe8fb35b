// lm_gemm.hpp -- the matrix-core tile product behind the linear cross entropy:
//   C[q][p] = sum_k P[p][k] Q[q][k],  BF16 operands, FP32 sums.
// P is the operand along a lane's four consecutive results (the dense side of
// C in memory), Q the one along its 16 lanes.  Each operand lies in memory
// either with its reduction index dense ([rows][k]) or as its transpose
// ([k][rows]); the second is turned around on the way from LDS to registers by
// the transposing LDS read, so no transposed copy is ever written.
//
// A workgroup owns a BM x BN tile of C and walks over k in steps of 64.  Both
// operands' tiles go from memory straight into LDS (16 bytes a lane, no
// registers in between), into one of two buffers while the other one is
// multiplied.  An LDS row's 16-byte pieces are permuted by an XOR with its row
// number, which is applied to the memory address a lane reads (a lane's place
// in LDS is fixed) and again when the fragments are read, so that the rows a
// fragment takes lie in different banks.  Lanes outside the operand read
// through a buffer descriptor at an offset beyond its end, which yields zeros.
#pragma once

#include "lm.hpp"

namespace lrs {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32acc_t __attribute__((ext_vector_type(4)));

// One operand: `rows` x `k` elements, `ld` elements between rows (or, where
// the reduction index is not the dense one, between reduction steps).
struct Operand {
    const void* p;
    int64_t ld;
    int rows;  // multiple of 8 where transposed (checked by the callers)
};

constexpr int GEMM_BK = 64;

// BM x BN tile, WM x WN waves; PT / QT: the operand lies as [k][rows].
template <int BM, int BN, int WM, int WN, bool PT, bool QT>
struct TileProduct {
    static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    static constexpr int P_BYTES = BM * GEMM_BK * 2, Q_BYTES = BN * GEMM_BK * 2, STAGE = P_BYTES + Q_BYTES;
    static constexpr int LDS_BYTES = 2 * STAGE;
    f32acc_t acc[FM][FN];

    // Bank spread of reduction step k in a transposed tile, in units of 32
    // bytes: the 16 steps a fragment read touches at once (4 of each 8 of 32)
    // use eight different ones.
    template <int R>
    static __device__ __forceinline__ int spread(int k) {
        return ((k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1);
    }

    // Loads of one operand's tile: R rows, this wave's share of R / 8 loads of 1 KiB.
    template <int R, bool TR>
    struct Loader {
        static constexpr int N = R / 8 / WAVES;
        static_assert(R / 8 % WAVES == 0, "loads divide over the waves");
        uint32_t off[N];   // byte offset of this lane's 16 bytes from the step's base
        int kfirst[N];     // its first reduction index within a step
        uint64_t base;
        int64_t step;
        __device__ __forceinline__ void init(const Operand& o, int row0, int k0) {
            const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const char* b = static_cast<const char*>(o.p);
            base = (uint64_t)(TR ? b + ((int64_t)k0 * o.ld + row0) * 2 : b + ((int64_t)row0 * o.ld + k0) * 2);
            step = TR ? GEMM_BK * o.ld * 2 : GEMM_BK * 2;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int L = wave + WAVES * j;
                if (TR) {
                    constexpr int PIECES = R / 8, KROWS = 64 / PIECES;  // 16-byte pieces of a step, steps of one load
                    const int k = L * KROWS + lane / PIECES;
                    const int col = ((lane % PIECES) ^ (spread<R>(k) * 2)) * 8;
                    off[j] = row0 + col < o.rows ? (uint32_t)((k * o.ld + col) * 2) : 0x80000000u;
                    kfirst[j] = k;
                } else {
                    const int r = 8 * L + lane / 8, piece = (lane % 8) ^ (lane / 8);
                    off[j] = row0 + r < o.rows ? (uint32_t)((r * o.ld + piece * 8) * 2) : 0x80000000u;
                    kfirst[j] = piece * 8;
                }
            }
        }
        // One load of 64 x 16 bytes into LDS at `to` (the wave's own KiB).  In
        // assembly, so that the compiler does not wait for it before the LDS
        // reads of the other buffer; it writes no register, and the wait
        // stands before the barrier that hands the buffer over.
        static __device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t o, const char* to) {
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                         :
                         : "s"((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)to), "v"(o), "s"(rsrc)
                         : "memory");
        }
        // requests the tile of one step into LDS; left: reduction indices left (64 or more, but in the last step)
        __device__ __forceinline__ void request(char* lds, int left) {
            const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, 0x7fffffff, 0x00020000);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint32_t o = left >= GEMM_BK || kfirst[j] < left ? off[j] : 0x80000000u;
                load_lds(rsrc, o, lds + (wave + WAVES * j) * 1024);
            }
            base += step;
        }
    };

    // Fragment f (16 rows from row f of the wave's first) of half kk of a step.
    template <int R, bool TR>
    struct Reader {
        static constexpr int MOST = R / 16 < 8 ? R / 16 : 8;  // fragments of a wave
        const char* at[TR ? MOST : 2];
        __device__ __forceinline__ void init(const char* tile, int row) {
            const int lane = threadIdx.x & 63;
            if (TR) {
                // lane s of 16 reads 4 columns of one of 4 steps and receives its own column of all four
                const int g = lane >> 4, s = lane & 15, k = 8 * g + (s >> 2);
#pragma unroll
                for (int i = 0; i < MOST; ++i)
                    at[i] = tile + k * (R * 2) + (((row / 16 + i) ^ spread<R>(k)) * 32) + (s & 3) * 8;
            } else {
                const int r = row + (lane & 15);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                    at[kk] = tile + r * 128 + (((lane >> 4) + 4 * kk) ^ (r & 7)) * 16;
            }
        }
        __device__ __forceinline__ bf16x8_t read(int f, int kk, int stage) const {
            typedef __attribute__((address_space(3))) s16x4_t lds4;
            if (TR) {
                const char* p = at[f] + kk * 32 * (R * 2) + stage;
                s16x4_t v[2];
                v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
                v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * (R * 2)));
                return __builtin_bit_cast(bf16x8_t, v);
            }
            return *reinterpret_cast<const bf16x8_t*>(at[kk] + f * 16 * 128 + stage);
        }
    };

    // First row of P and of Q that this wave's fragments start at.
    static __device__ __forceinline__ int wave_p() { return (int)(threadIdx.x >> 6) / WN * (BM / WM); }
    static __device__ __forceinline__ int wave_q() { return (int)(threadIdx.x >> 6) % WN * (BN / WN); }

    __device__ __forceinline__ void run(char* lds, const Operand& p, const Operand& q, int p0, int q0, int k0, int k1) {
        Loader<BM, PT> lp;
        Loader<BN, QT> lq;
        Reader<BM, PT> rp;
        Reader<BN, QT> rq;
        lp.init(p, p0, k0);
        lq.init(q, q0, k0);
        rp.init(lds, wave_p());
        rq.init(lds + P_BYTES, wave_q());
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32acc_t{0.f, 0.f, 0.f, 0.f};
        lp.request(lds, k1 - k0);
        lq.request(lds + P_BYTES, k1 - k0);
        int stage = 0;
        for (int k = k0; k < k1; k += GEMM_BK) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (k + GEMM_BK < k1) {
                lp.request(lds + (STAGE - stage), k1 - k - GEMM_BK);
                lq.request(lds + (STAGE - stage) + P_BYTES, k1 - k - GEMM_BK);
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8_t a[FM], b[FN];
#pragma unroll
                for (int i = 0; i < FM; ++i) a[i] = rp.read(i, kk, stage);
#pragma unroll
                for (int j = 0; j < FN; ++j) b[j] = rq.read(j, kk, stage);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
            }
            stage = STAGE - stage;
        }
        __syncthreads();
    }
};

}  // namespace lrs
