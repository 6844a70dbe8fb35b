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
// registers in between).  An LDS row's 16-byte pieces are permuted by an XOR
// with its row number, which is applied to the memory address a lane reads (a
// lane's place in LDS is fixed) and again when the fragments are read, so that
// the rows a fragment takes lie in different banks (no conflict is counted in the forward, dh and dw; dz's end, where
// each lane reads its tokens from LDS, counts 10^5 over 1000 workgroups).
// Lanes outside the operand read through a buffer descriptor at an offset
// beyond its end, which yields zeros.
//
// TileProduct halves each operand's tile and orders a step as four phases, one
// a pair of halves, so that every phase multiplies what stands in registers while
// the half that the next phase needs is read from LDS and the same half of the step
// after the next is loaded into the place that was read last: the loads have one
// to two steps to arrive, two barriers a step hand places over, and the second
// step's Q halves come in the other order so that no fragment is read twice.
//
// What bounds it (256 x 256, long k, random data): the power budget.  From
// registers alone the matrix cores run at 2.39 PFLOP/s on zeros and 2.02 on
// random data; with LDS and memory the clock settles at 1.9 to 2.1 GHz and the
// products run at 1.3 to 1.4 PFLOP/s, 56 to 68% of the cycles on the matrix cores (a
// library product of 8192 x 2048 x 128000: 1.40).  Measured on the way (dw of 8192 x 2048
// x 128000, eight chunks): one read-multiply-barrier loop 448 us a chunk; the reads of
// one half step under the products of the other 423; phases with few scalar
// instructions a load and 8 waves 408, with 4 waves of 128 x 128, which
// read a third less LDS, 375.  With 4 waves the sums stand in
// accumulation registers through products written in assembly: left to the
// compiler they moved and spilled (1430 us).  A workgroup that runs on to its next tile
// with that tile's first loads in flight changed nothing (13.2 against 13.0 ms).
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

// A barrier for what the workgroup keeps in LDS, which leaves loads and stores in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// BM x BN tile, WM x WN waves; PT / QT: the operand lies as [k][rows].
template <int BM, int BN, int WM, int WN, bool PT, bool QT>
struct TileProduct {
    static constexpr int WAVES = WM * WN, THREADS = WAVES * 64, TILE_P = BM, TILE_Q = BN, WAVES_P = WM;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;          // fragments of a wave
    static constexpr int HP = BM / 2, HQ = BN / 2, HM = FM / 2, HN = FN / 2;  // and of a half: rows, fragments of a wave
    static constexpr bool ROOMY = WAVES == 4;  // one wave a SIMD: 512 registers
    static constexpr int STAGE = (BM + BN) * GEMM_BK * 2, LDS_BYTES = 2 * STAGE;
    f32acc_t acc[FM][FN];

    // Bank spread of reduction step k in a transposed half of R rows, in units
    // of 32 bytes: the 16 steps that a fragment read touches at once (4 of each 8
    // of 32) lie on all eight 32-byte groups of the 64 banks, twice each.
    template <int R>
    static __device__ __forceinline__ int spread(int k) {
        static_assert(R == 128 || R == 64, "256 or 128 bytes a step");
        return R == 128 ? (k & 3) | ((k >> 3) & 1) << 2 : ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
    }

    // Loads of an operand's tile, half by half: R rows a half, this wave's share of R / 8 loads of 1 KiB.
    template <int R, bool TR>
    struct Loader {
        static constexpr int N = R / 8 / WAVES;
        static_assert(R / 8 % WAVES == 0, "loads divide over the waves");
        uint32_t off[2][N];  // byte offset of this lane's 16 bytes from the step's base
        int piece;           // first reduction index of those 16 bytes within a step (where it is dense)
        uint64_t base;
        int64_t step;
        uint32_t line;       // bytes from one reduction index to the next (where it is not dense)
        int left;            // reduction indices from this step on
        uint32_t to;         // LDS address of this wave's first load
        __device__ __forceinline__ void init(const char* lds, const Operand& o, int row0, int k0, int k1) {
            const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const char* b = static_cast<const char*>(o.p);
            base = (uint64_t)(TR ? b + ((int64_t)k0 * o.ld + row0) * 2 : b + ((int64_t)row0 * o.ld + k0) * 2);
            step = TR ? GEMM_BK * o.ld * 2 : GEMM_BK * 2;
            line = (uint32_t)(o.ld * 2);
            left = k1 - k0;
            piece = ((lane % 8) ^ (lane / 8)) * 8;
            to = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)lds + wave * 1024;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int L = wave + WAVES * j;
                    if (TR) {
                        constexpr int PIECES = R / 8, KROWS = 64 / PIECES;  // 16-byte pieces of a step, steps of one load
                        const int k = L * KROWS + lane / PIECES;
                        const int col = h * R + ((lane % PIECES) ^ (spread<R>(k) * 2)) * 8;
                        off[h][j] = row0 + col < o.rows ? (uint32_t)((k * o.ld + col) * 2) : 0x80000000u;
                    } else {
                        const int r = h * R + 8 * L + lane / 8;
                        off[h][j] = row0 + r < o.rows ? (uint32_t)((r * o.ld + piece) * 2) : 0x80000000u;
                    }
                }
        }
        // Requests load j of half h of the step, 64 x 16 bytes into LDS at `at`
        // from this wave's place; beyond the last reduction index it writes zeros
        // (past the descriptor's end, or, where the index is dense, lane by lane).
        // In assembly, so that the compiler does not wait for it before the
        // LDS reads of the other halves; it writes no register, and the
        // wait stands before the barrier that hands the half over.
        __device__ __forceinline__ void request(int at, int h, int j) {
            const int some = left < 0 ? 0 : left < GEMM_BK ? left : GEMM_BK;
            const uint32_t end = TR ? (uint32_t)__builtin_amdgcn_readfirstlane((int)(some * line)) : 0x7fffffffu;
            const u32x4_t rsrc = {(uint32_t)base, (uint32_t)(base >> 32), end, 0x00020000u};
            const uint32_t o = TR || piece < some ? off[h][j] : 0x80000000u;
            asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
                         :
                         : "s"(to), "s"(at + WAVES * 1024 * j), "v"(o), "s"(rsrc)
                         : "memory", "scc", "m0");
        }
        __device__ __forceinline__ void request_half(int at, int h) {
#pragma unroll
            for (int j = 0; j < N; ++j) request(at, h, j);
        }
        __device__ __forceinline__ void advance() {
            base += step;
            left -= GEMM_BK;
        }
    };

    // Fragment f (16 rows) of this wave's rows in a half, steps 32 kk to 32 kk + 31.
    template <int R, bool TR>
    struct Reader {
        uint32_t at[TR ? 1 : 2];  // LDS addresses
        __device__ __forceinline__ void init(const char* tile, int row) {
            const int lane = threadIdx.x & 63;
            const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)tile;
            if constexpr (TR) {
                // lane s of 16 reads 4 columns of one of 4 steps and receives its own column of all four
                const int g = lane >> 4, s = lane & 15, k = 8 * g + (s >> 2);
                at[0] = lds + k * (R * 2) + (((row / 16) ^ spread<R>(k)) * 32) + (s & 3) * 8;
            } else {
                const int r = row + (lane & 15);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                    at[kk] = lds + r * 128 + (((lane >> 4) + 4 * kk) ^ (r & 7)) * 16;
            }
        }
        __device__ __forceinline__ bf16x8_t read(int f, int kk, int from) const {
            typedef __attribute__((address_space(3))) s16x4_t lds4;
            typedef __attribute__((address_space(3))) bf16x8_t lds8;
            // With two waves a SIMD the address is formed where it is used: kept over the
            // loop, those of all fragments and stages would not fit the registers.
            uint32_t o = at[TR ? 0 : kk];
            if (!ROOMY) asm volatile("" : "+v"(o));
            if constexpr (TR) {  // f is below the power of two that divides the wave's first fragment: an XOR adds it
                o = (o ^ (uint32_t)(f * 32)) + (uint32_t)(kk * 32 * (R * 2) + from);
                s16x4_t v[2];
                v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)o);
                v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(o + 4 * (R * 2)));
                return __builtin_bit_cast(bf16x8_t, v);
            } else {
                return *(const lds8*)(o + (uint32_t)(f * 16 * 128 + from));
            }
        }
    };

    // Row of the tile that fragment i of P (j of Q) of this wave starts at.
    static __device__ __forceinline__ int row_p(int i) {
        return i / HM * HP + (int)(threadIdx.x >> 6) / WN * (HM * 16) + i % HM * 16;
    }
    static __device__ __forceinline__ int row_q(int j) {
        return j / HN * HQ + (int)(threadIdx.x >> 6) % WN * (HN * 16) + j % HN * 16;
    }

    // Byte offsets within a stage of half h of P and of Q.
    static constexpr int at_p(int h) { return h * HP * GEMM_BK * 2; }
    static constexpr int at_q(int h) { return BM * GEMM_BK * 2 + h * HQ * GEMM_BK * 2; }

    struct State {
        Loader<HP, PT> lp;
        Loader<HQ, QT> lq;
        Reader<HP, PT> rp;
        Reader<HQ, QT> rq;
        bf16x8_t a[2][HM][2], b[2][HN][2];  // fragments of each half: [half][fragment][kk]
    };
    static constexpr int LOADS = Loader<HP, PT>::N;
    static_assert(LOADS == Loader<HQ, QT>::N, "a half of either operand is as many loads");

    // One of four phases of a step: the products of half X of P and Y of Q.
    // Between them stand the reads of the half that comes next (half RH of P
    // or Q, at `from`) and loads of the step after the next (half LH, to `to`), so that neither
    // the matrix cores nor the queues of LDS and memory wait for each other.
    template <int X, int Y, bool READ_P, int RH, bool LOAD_P, int LH>
    __device__ __forceinline__ void phase(State& s, int from, int to) {
        constexpr int M = HM * HN * 2, READS = 2 * (READ_P ? HM : HN);
#pragma unroll
        for (int t = 0; t < M; ++t) {
#pragma unroll
            for (int r = 0; r < READS; ++r)
                if (r * (M / 2) / READS == t) {
                    if (READ_P) s.a[RH][r / 2][r % 2] = s.rp.read(r / 2, r % 2, from + at_p(RH));
                    else s.b[RH][r / 2][r % 2] = s.rq.read(r / 2, r % 2, from + at_q(RH));
                }
#pragma unroll
            for (int l = 0; l < LOADS; ++l)
                if (l * M / LOADS + 1 == t) {
                    if (LOAD_P) s.lp.request(to + at_p(LH), LH, l);
                    else s.lq.request(to + at_q(LH), LH, l);
                }
            __builtin_amdgcn_sched_barrier(0);
            const int kk = t / (HM * HN), i = t / HN % HM, j = t % HN;
            f32acc_t& c = acc[X * HM + i][Y * HN + j];
            if (ROOMY) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(s.a[X][i][kk]), "v"(s.b[Y][j][kk]));
            else c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(s.a[X][i][kk], s.b[Y][j][kk], c, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // What the two phases before read is in registers, so that its place can be
    // loaded again, and what the next two read (requested three pairs of phases
    // ago) has landed.
    static __device__ __forceinline__ void hand_over() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(4 * LOADS) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }

    // Step whose first half of Q is F; its buffers are those of `stage`.
    template <int F>
    __device__ __forceinline__ void step(State& s) {
        constexpr int stage = F * STAGE;
        phase<0, F, false, 1 - F, true, 0>(s, stage, stage);
        phase<0, 1 - F, true, 1, false, F>(s, stage, stage);
        hand_over();
        phase<1, 1 - F, true, 0, false, 1 - F>(s, STAGE - stage, stage);
        s.lq.advance();
        phase<1, F, false, 1 - F, true, 1>(s, STAGE - stage, stage);
        s.lp.advance();
        hand_over();
    }

    __device__ __forceinline__ void run(char* lds, const Operand& p, const Operand& q, int p0, int q0, int k0, int k1) {
        State s;
        s.lp.init(lds, p, p0, k0, k1);
        s.lq.init(lds, q, q0, k0, k1);
        s.rp.init(lds, row_p(0));
        s.rq.init(lds, row_q(0));
        // steps 0 and 1 in the order in which they are read
        s.lp.request_half(at_p(0), 0);
        s.lq.request_half(at_q(0), 0);
        s.lq.request_half(at_q(1), 1);
        s.lp.request_half(at_p(1), 1);
        s.lp.advance();
        s.lq.advance();
        s.lp.request_half(STAGE + at_p(0), 0);
        s.lq.request_half(STAGE + at_q(1), 1);
        s.lq.request_half(STAGE + at_q(0), 0);
        s.lp.request_half(STAGE + at_p(1), 1);
        s.lp.advance();
        s.lq.advance();
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32acc_t{0.f, 0.f, 0.f, 0.f};
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(6 * LOADS) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int j = 0; j < HN; ++j) s.b[0][j][kk] = s.rq.read(j, kk, at_q(0));
#pragma unroll
            for (int i = 0; i < HM; ++i) s.a[0][i][kk] = s.rp.read(i, kk, at_p(0));
        }
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(4 * LOADS) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // two steps at a time; where their number is odd the last is one of zeros
        for (int k = k0; k < k1; k += 2 * GEMM_BK) {
            step<0>(s);
            step<1>(s);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (ROOMY) asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
    }
};

// The same product for tiles of few rows, where a wave has too few fragments to
// halve: the next step's tile is loaded while one step is multiplied.
template <int BM, int BN, int WM, int WN, bool PT, bool QT>
struct ThinProduct {
    static constexpr int WAVES = WM * WN, THREADS = WAVES * 64, TILE_P = BM, TILE_Q = BN, WAVES_P = WM;
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
                         : "memory", "m0");
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
    static __device__ __forceinline__ int row_p(int i) { return wave_p() + 16 * i; }
    static __device__ __forceinline__ int row_q(int j) { return wave_q() + 16 * j; }

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
