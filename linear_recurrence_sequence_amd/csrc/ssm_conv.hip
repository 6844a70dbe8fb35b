// ssm_conv.hip -- the short causal convolution of each channel over time,
// forward, backward and for single tokens.
//
//   p_t = bias + sum_{j < W} w[W-1-j] x_{t-j},  y = act(p);
//   g = dy act'(p),  dx_t = sum_j w[W-1-j] g_{t+j},  dw[W-1-j] = sum_t g_t x_{t-j},  dbias = sum_t g_t.
//
// Bound by memory: a lane holds four channels and walks over a piece of a row with the last W - 1 inputs in registers,
// so that each input is read once but for the W - 1 tokens before a piece (and behind it, backward).  The backward
// walks the same way: the g of a token is added to the dx of the W tokens that it came from, which are stored one after
// the other as they are complete.  A sequence's start clears what is held.
//
// 32768 x 2560 in BF16 with SiLU, packed: forward 64 us, 5.3 TB/s; backward 126 us, 4.0 TB/s, and 13 us for the sums (a copy of the same input takes 60 us, a sum of
// two tensors 86).  In FP32 129 us, and 349 with the sums, with three taps 213: the four-tap backward spills 9 to 12 of its 128 registers there.
// Four channels a lane forward, two backward, whose sums and cotangents would else take 200 registers (235 us).
#include "lm.hpp"
#include "ssm_lay.hpp"

namespace lrs {
namespace {

// Tokens of a block, whose loads are in flight together while the block before is worked on: waves start together, and would else all
// wait, then all compute.
constexpr int AHEAD = 4;

// V consecutive channels of a row, at a lane's first channel `col` below d; TAIL: d is no multiple of V.
template <class T, int V, bool TAIL>
struct Cols;
template <class T, bool TAIL>
struct Cols<T, 4, TAIL> {
    Quad<T> q;
    static __device__ __forceinline__ Cols load(const T* row, int col, int d) { return {row_load<T, TAIL>(row, col, d)}; }
    static __device__ __forceinline__ Cols zero() { return {Quad<T>::zero()}; }
    __device__ __forceinline__ void get(int col, int d, float* f) const { take<TAIL>(q, col, d, f); }
    static __device__ __forceinline__ void store(T* row, int col, int d, const float* f) { row_store<T, TAIL>(row, col, d, f); }
};
template <class T, bool TAIL>
struct Cols<T, 2, TAIL> {
    Pair<T> q;
    // the channel that a row ends in is loaded as the second of a pair
    static __device__ __forceinline__ Cols load(const T* row, int col, int d) {
        if (TAIL && d == 1) return {Pair<T>::one(row)};
        return {Pair<T>::load(reinterpret_cast<const char*>(row + (TAIL ? min(col, d - 2) : col)), 0)};
    }
    static __device__ __forceinline__ Cols zero() { return {Pair<T>{}}; }
    __device__ __forceinline__ void get(int col, int d, float* f) const {
        const float2 v = q.get();
        const bool last = TAIL && col == d - 1;
        f[0] = last ? v.y : v.x, f[1] = last ? 0.0f : v.y;
    }
    static __device__ __forceinline__ void store(T* row, int col, int d, const float* f) {
        store_pair<T>(reinterpret_cast<char*>(row + col), 0, make_float2(f[0], f[1]), true, !TAIL || col + 1 < d);
    }
};

// Which channels and tokens a thread has.
struct Walk {
    int col, b, piece, t0, t1, len;
    bool on;
};
template <int V>
__device__ __forceinline__ Walk walk_of(const ConvArgs& a) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, lanes = (a.d + V - 1) / V, unit = x / lanes;
    Walk k;
    k.on = unit < (int64_t)a.batch * a.pieces;
    k.col = V * (int)(x % lanes);
    k.b = (int)(unit / a.pieces);
    k.piece = (int)(unit % a.pieces);
    k.t0 = k.piece * a.tokens;
    k.t1 = min(k.t0 + a.tokens, a.length);
    k.len = !k.on ? 0 : a.lengths ? min(max(a.lengths[k.b], 0), a.length) : a.length;
    return k;
}

template <class T, int W, int V, bool TAIL>
struct Conv {
    float w[W][V], bias[V];
    float x[W][V];                              // x[0] the newest input

    __device__ __forceinline__ void load(const ConvArgs& a, int col) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = min(col + i, a.d - 1);
            bias[i] = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = a.w[(int64_t)c * W + k];
        }
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) x[k][i] = 0.0f;
    }
    // A token's input as the next one; a sequence's start forgets the others.
    template <bool STARTS = true>
    __device__ __forceinline__ void push(const float* v, bool start) {
#pragma unroll
        for (int k = W - 1; k > 0; --k)
#pragma unroll
            for (int i = 0; i < V; ++i) x[k][i] = STARTS && start ? 0.0f : x[k - 1][i];
#pragma unroll
        for (int i = 0; i < V; ++i) x[0][i] = v[i];
    }
    // The inputs of the W - 1 tokens before t (padding counts as zero).
    __device__ __forceinline__ void before(const ConvArgs& a, int b, int col, int t, int len) {
        Cols<T, V, TAIL> q[W - 1];
        bool start[W - 1];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int s = t - (W - 1) + k;
            const int64_t row = (int64_t)b * a.length + s;
            start[k] = s >= 0 && a.reset && a.reset[row] != 0;
            if (s >= 0 && s < len) q[k] = Cols<T, V, TAIL>::load(static_cast<const T*>(a.x) + row * a.x_stride, col, a.d);
            else if (s < 0 && a.state) q[k] = Cols<T, V, TAIL>::load(static_cast<const T*>(a.state) + ((int64_t)b * (W - 1) + s + W - 1) * a.d, col, a.d);
            else q[k] = Cols<T, V, TAIL>::zero();
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float v[V];
            q[k].get(col, a.d, v);
            push(v, start[k]);
        }
    }
    __device__ __forceinline__ void sum(float* p) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = bias[i];
#pragma unroll
            for (int k = W - 1; k >= 0; --k) p[i] = fmaf(w[W - 1 - k][i], x[k][i], p[i]);
        }
    }
};

template <class T, int W, int V, bool TAIL>
__global__ __launch_bounds__(256) void conv_fwd_kernel(const ConvArgs a) {
    const Walk k = walk_of<V>(a);
    if (!k.on) return;
    Conv<T, W, V, TAIL> c;
    c.load(a, k.col);
    if (k.piece == 0 && a.state_out) {          // the inputs before the row's end
        c.before(a, k.b, k.col, k.len, k.len);
        T* to = static_cast<T*>(a.state_out) + (int64_t)k.b * (W - 1) * a.d;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) Cols<T, V, TAIL>::store(to + (int64_t)(W - 2 - i) * a.d, k.col, a.d, c.x[i]);
    }
    if (k.t0 >= a.length) return;
    c.before(a, k.b, k.col, k.t0, k.len);
    const int64_t row0 = (int64_t)k.b * a.length;
    Cols<T, V, TAIL> next[AHEAD];
    uint8_t flags[AHEAD] = {};                   // as loaded: joined here, they would be waited for before the block is due
    const auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t row = row0 + min(t0 + i, a.length - 1);
            next[i] = Cols<T, V, TAIL>::load(static_cast<const T*>(a.x) + row * a.x_stride, k.col, a.d);
            if (a.reset) flags[i] = a.reset[row];
        }
    };
    fetch(k.t0);
    for (int t0 = k.t0; t0 < k.t1; t0 += AHEAD) {
        Cols<T, V, TAIL> q[AHEAD];
        uint32_t start = 0;                      // bit i: the block's token i starts a sequence
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) q[i] = next[i], start |= (flags[i] != 0) << i;
        if (t0 + AHEAD < k.t1) fetch(t0 + AHEAD);
        const bool any = t0 + AHEAD > min(k.t1, k.len) || start;
        both_ways(__any(any), [&](auto some) {  // some: of the wave's tokens start a sequence, or are padding, or behind its piece
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int t = t0 + i;
                float v[V], y[V];
                q[i].get(k.col, a.d, v);
                c.template push<decltype(some)::value>(v, start >> i & 1);
                c.sum(y);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (a.act) y[e] *= sigmoid_of(y[e]);
                    if (decltype(some)::value) y[e] = t < k.len ? y[e] : 0.0f;  // padding: whatever x holds
                }
                if (!decltype(some)::value || t < k.t1) Cols<T, V, TAIL>::store(static_cast<T*>(a.y) + (row0 + t) * a.d, k.col, a.d, y);
            }
        });
    }
}

template <class T, int W, int V, bool TAIL>
__global__ __launch_bounds__(256, V == 2 ? 4 : 1) void conv_bwd_kernel(const ConvArgs a) {
    const Walk k = walk_of<V>(a);
    if (!k.on) return;
    Conv<T, W, V, TAIL> c;
    c.load(a, k.col);
    c.before(a, k.b, k.col, k.t0, k.len);
    float dw[W][V], db[V], dx[W][V];            // dx[j]: of the token j before the newest
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = dx[j][i] = 0.0f;
    }
    const int64_t row0 = (int64_t)k.b * a.length;
    int since = W;                               // tokens since a sequence's start
    Cols<T, V, TAIL> next[2][AHEAD];             // x, dy
    uint8_t flags[AHEAD] = {};
    const auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t row = row0 + max(min(t0 + i, a.length - 1), 0);
            if (a.length > 0) {
                next[0][i] = Cols<T, V, TAIL>::load(static_cast<const T*>(a.x) + row * a.x_stride, k.col, a.d);
                next[1][i] = Cols<T, V, TAIL>::load(static_cast<const T*>(a.dy) + row * a.dy_stride, k.col, a.d);
                if (a.reset) flags[i] = a.reset[row];
            } else {
                next[0][i] = next[1][i] = Cols<T, V, TAIL>::zero();
            }
        }
    };
    fetch(k.t0);
    // the W - 1 tokens behind the piece are formed for the dx of its last ones
    for (int t0 = k.t0; t0 < k.t1 + W - 1; t0 += AHEAD) {
        Cols<T, V, TAIL> q[AHEAD], r[AHEAD];
        uint32_t start = 0;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) q[i] = next[0][i], r[i] = next[1][i], start |= (flags[i] != 0 && t0 + i < k.len) << i;
        if (t0 + AHEAD < k.t1 + W - 1) fetch(t0 + AHEAD);
        // a token that needs more than the plain sums: a start, padding, what is behind the piece, or whose dx has a part from the state
        const bool any = t0 + AHEAD > min(k.t1, k.len) || t0 - (W - 1) < k.t0 || (a.dstate_out && t0 + AHEAD > k.len - (W - 1)) || since < W || start;
        both_ways(__any(any), [&](auto more) {
            constexpr bool MORE = decltype(more)::value;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int t = t0 + i;
                float v[V], g[V], p[V];
                q[i].get(k.col, a.d, v);
                r[i].get(k.col, a.d, g);
                const bool in = t < k.len;
                if (MORE) {
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] = in ? v[e] : 0.0f;
                    since = start >> i & 1 ? 0 : min(since + 1, W);
                }
                c.template push<MORE>(v, start >> i & 1);
                c.sum(p);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (a.act) {
                        const float s = sigmoid_of(p[e]);
                        g[e] *= s * fmaf(p[e], 1.0f - s, 1.0f);
                    }
                    if (MORE) g[e] = in ? g[e] : 0.0f;
                    const float mine = !MORE || t < k.t1 ? g[e] : 0.0f;  // of the tokens behind, dx alone is this piece's
                    db[e] += mine;
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[W - 1 - j][e] = fmaf(mine, c.x[j][e], dw[W - 1 - j][e]);
#pragma unroll
                    for (int j = W - 1; j >= 0; --j)
                        dx[j][e] = fmaf(c.w[W - 1 - j][e], !MORE || since >= j ? g[e] : 0.0f, j ? dx[j - 1][e] : 0.0f);
                    // here and now: put off to the block's end, these sums would keep all of its inputs in registers
                    asm volatile("" : "+v"(db[e]));
#pragma unroll
                    for (int j = 0; j < W; ++j) asm volatile("" : "+v"(dw[j][e]));
                }
                const int done = t - (W - 1);    // the token that no later one reaches
                if (MORE) {
                    const int late = done - (k.len - (W - 1));
                    if (late >= 0 && late < W - 1 && a.dstate_out && done < a.length) {
                        bool kept = true;        // its input is in the state that the row leaves
                        for (int s = max(done + 1, 0); s < k.len; ++s) kept = kept && !(a.reset && a.reset[row0 + s] != 0);
                        if (kept) {
                            float o[V];
                            const T* from = static_cast<const T*>(a.dstate_out) + ((int64_t)k.b * (W - 1) + late) * a.d;
                            Cols<T, V, TAIL>::load(from, k.col, a.d).get(k.col, a.d, o);
#pragma unroll
                            for (int e = 0; e < V; ++e) dx[W - 1][e] += o[e];
                        }
                    }
                }
                if (!MORE || (done >= k.t0 && done < k.t1))
                    Cols<T, V, TAIL>::store(static_cast<T*>(a.dx) + (row0 + done) * a.d, k.col, a.d, dx[W - 1]);
                else if (done < 0 && k.piece == 0 && a.dstate)
                    Cols<T, V, TAIL>::store(static_cast<T*>(a.dstate) + ((int64_t)k.b * (W - 1) + done + W - 1) * a.d, k.col, a.d, dx[W - 1]);
            }
        });
    }
    float* part = a.part + ((int64_t)k.b * a.pieces + k.piece) * (W + 1) * a.d;
#pragma unroll
    for (int j = 0; j < W; ++j) Cols<float, V, TAIL>::store(part + (int64_t)j * a.d, k.col, a.d, dw[j]);
    Cols<float, V, TAIL>::store(part + (int64_t)W * a.d, k.col, a.d, db);
}

// dw and dbias over the pieces, FP64 in a fixed order: 16 channels a workgroup, 64 lanes down each.  blockIdx.y: a tap, or the bias.
__global__ __launch_bounds__(1024) void conv_join_kernel(const float* part, int64_t parts, int d, int width, float* dw, float* dbias) {
    __shared__ double buf[16][17];
    const int c = threadIdx.x & 15, lane = threadIdx.x >> 4, col = blockIdx.x * 16 + c, k = blockIdx.y;
    double s = 0.0;
    if (col < d)
        for (int64_t i = lane; i < parts; i += 64 * 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = i + 64 * u < parts ? part[((i + 64 * u) * (width + 1) + k) * d + col] : 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) s += (double)v[u];
        }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if ((lane & 3) == 0) buf[lane >> 2][c] = s;
    __syncthreads();
    if (lane == 0 && col < d) {
        double v = buf[0][c];
#pragma unroll
        for (int i = 1; i < 16; ++i) v += buf[i][c];
        if (k < width) dw[(int64_t)col * width + k] = (float)v;
        else if (dbias) dbias[col] = (float)v;
    }
}

// One token: a thread has four channels of a sequence.  (Where d is no multiple of 4 the last thread of a row also loads elements that
// its neighbour may have moved on already; it uses none of them.)
template <class T, int W, int V, bool TAIL>
__global__ __launch_bounds__(256) void conv_step_kernel(const ConvArgs a) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, lanes = (a.d + V - 1) / V, b = x / lanes;
    const int col = V * (int)(x % lanes);
    if (b >= a.batch) return;
    Conv<T, W, V, TAIL> c;
    Cols<T, V, TAIL> q[W];
    T* st = static_cast<T*>(const_cast<void*>(a.state)) + b * (W - 1) * a.d;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) q[k] = Cols<T, V, TAIL>::load(st + (int64_t)k * a.d, col, a.d);
    q[W - 1] = Cols<T, V, TAIL>::load(static_cast<const T*>(a.x) + b * a.x_stride, col, a.d);
    c.load(a, col);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        float v[V];
        q[k].get(col, a.d, v);
        c.push(v, false);
    }
    float y[V];
    c.sum(y);
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (a.act) y[e] *= sigmoid_of(y[e]);
    Cols<T, V, TAIL>::store(static_cast<T*>(a.y) + b * a.d, col, a.d, y);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) Cols<T, V, TAIL>::store(st + (int64_t)k * a.d, col, a.d, c.x[W - 2 - k]);
}

enum Kind { FWD, BWD, STEP };
// Channels of a lane.
constexpr int FWD_V = 4, BWD_V = 2, STEP_V = 4;
template <Kind K, class T, int W, bool TAIL>
void launch_one(const ConvArgs& a, hipStream_t s) {
    constexpr int V = K == FWD ? FWD_V : K == BWD ? BWD_V : STEP_V;
    const int64_t threads = ceil_div(a.d, V) * a.batch * (K == STEP ? 1 : a.pieces);
    const dim3 g((unsigned)ceil_div(threads, 256)), b(256);
    if constexpr (K == FWD) LRS_LAUNCH(K_CONV, (conv_fwd_kernel<T, W, V, TAIL>), g, b, 0, s, a);
    else if constexpr (K == BWD) LRS_LAUNCH(K_CONV_BWD, (conv_bwd_kernel<T, W, V, TAIL>), g, b, 0, s, a);
    else LRS_LAUNCH(K_CONV_STEP, (conv_step_kernel<T, W, V, TAIL>), g, b, 0, s, a);
}
template <Kind K, class T, int W>
void launch_tail(const ConvArgs& a, hipStream_t s) {
    constexpr int V = K == FWD ? FWD_V : K == BWD ? BWD_V : STEP_V;
    if (a.d % V) launch_one<K, T, W, true>(a, s);
    else launch_one<K, T, W, false>(a, s);
}
template <Kind K, class T>
void launch_width(const ConvArgs& a, hipStream_t s) {
    if (a.width == 2) launch_tail<K, T, 2>(a, s);
    else if (a.width == 3) launch_tail<K, T, 3>(a, s);
    else launch_tail<K, T, 4>(a, s);
}
template <Kind K>
hipError_t launch(const ConvArgs& a, bool f32, hipStream_t s) {
    if (f32) launch_width<K, float>(a, s);
    else launch_width<K, uint16_t>(a, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs& a, bool f32, hipStream_t s) { return launch<FWD>(a, f32, s); }
hipError_t launch_conv_step(const ConvArgs& a, bool f32, hipStream_t s) { return launch<STEP>(a, f32, s); }
hipError_t launch_conv_bwd(const ConvArgs& a, bool f32, hipStream_t s) {
    if (a.batch > 0) {
        const hipError_t e = launch<BWD>(a, f32, s);
        if (e != hipSuccess) return e;
    }
    LRS_LAUNCH(K_CONV_JOIN, conv_join_kernel, dim3((unsigned)ceil_div(a.d, 16), a.width + 1), dim3(1024), 0, s, (const float*)a.part,
               (int64_t)a.batch * a.pieces, a.d, a.width, a.dw, a.dbias);
    return hipGetLastError();
}

}  // namespace lrs
