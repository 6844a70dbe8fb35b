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
#include "lm.hpp"
#include "ssm.hpp"

namespace lrs {
namespace {

constexpr int AHEAD = 8;  // tokens whose loads are in flight together

// Which channels and tokens a thread has.
struct Walk {
    int col, b, piece, t0, t1, len;
    bool on;
};
__device__ __forceinline__ Walk walk_of(const ConvArgs& a) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, quads = (a.d + 3) / 4, unit = x / quads;
    Walk k;
    k.on = unit < (int64_t)a.batch * a.pieces;
    k.col = 4 * (int)(x % quads);
    k.b = (int)(unit / a.pieces);
    k.piece = (int)(unit % a.pieces);
    k.t0 = k.piece * a.tokens;
    k.t1 = min(k.t0 + a.tokens, a.length);
    k.len = !k.on ? 0 : a.lengths ? min(max(a.lengths[k.b], 0), a.length) : a.length;
    return k;
}

template <class T, int W, bool TAIL>
struct Conv {
    float w[W][4], bias[4];
    float x[W][4];                              // x[0] the newest input

    __device__ __forceinline__ void load(const ConvArgs& a, int col) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = min(col + i, a.d - 1);
            bias[i] = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][i] = a.w[(int64_t)c * W + k];
        }
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[k][i] = 0.0f;
    }
    // A token's input as the next one; a sequence's start forgets the others.
    __device__ __forceinline__ void push(const float* v, bool start) {
#pragma unroll
        for (int k = W - 1; k > 0; --k)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[k][i] = start ? 0.0f : x[k - 1][i];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[0][i] = v[i];
    }
    // The inputs of the W - 1 tokens before t (padding counts as zero).
    __device__ __forceinline__ void before(const ConvArgs& a, int b, int col, int t, int len) {
        Quad<T> q[W - 1];
        bool start[W - 1];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int s = t - (W - 1) + k;
            const int64_t row = (int64_t)b * a.length + s;
            start[k] = s >= 0 && a.reset && a.reset[row] != 0;
            if (s >= 0 && s < len) q[k] = row_load<T, TAIL>(static_cast<const T*>(a.x) + row * a.x_stride, col, a.d);
            else if (s < 0 && a.state) q[k] = row_load<T, TAIL>(static_cast<const T*>(a.state) + ((int64_t)b * (W - 1) + s + W - 1) * a.d, col, a.d);
            else q[k] = Quad<T>::zero();
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float v[4];
            take<TAIL>(q[k], col, a.d, v);
            push(v, start[k]);
        }
    }
    __device__ __forceinline__ void sum(float* p) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[i] = bias[i];
#pragma unroll
            for (int k = W - 1; k >= 0; --k) p[i] = fmaf(w[W - 1 - k][i], x[k][i], p[i]);
        }
    }
};

template <class T, int W, bool TAIL>
__global__ __launch_bounds__(256) void conv_fwd_kernel(const ConvArgs a) {
    const Walk k = walk_of(a);
    if (!k.on) return;
    Conv<T, W, TAIL> c;
    c.load(a, k.col);
    if (k.piece == 0 && a.state_out) {          // the inputs before the row's end
        c.before(a, k.b, k.col, k.len, k.len);
        T* to = static_cast<T*>(a.state_out) + (int64_t)k.b * (W - 1) * a.d;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) row_store<T, TAIL>(to + (int64_t)(W - 2 - i) * a.d, k.col, a.d, c.x[i]);
    }
    if (k.t0 >= a.length) return;
    c.before(a, k.b, k.col, k.t0, k.len);
    const int64_t row0 = (int64_t)k.b * a.length;
    for (int t0 = k.t0; t0 < k.t1; t0 += AHEAD) {
        Quad<T> q[AHEAD];
        bool start[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t row = row0 + min(t0 + i, a.length - 1);
            q[i] = row_load<T, TAIL>(static_cast<const T*>(a.x) + row * a.x_stride, k.col, a.d);
            start[i] = a.reset && a.reset[row] != 0;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int t = t0 + i;
            float v[4], y[4];
            take<TAIL>(q[i], k.col, a.d, v);
            c.push(v, start[i]);
            c.sum(y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (a.act) y[e] *= sigmoid_of(y[e]);
                y[e] = t < k.len ? y[e] : 0.0f;  // padding: whatever x holds
            }
            if (t < k.t1) row_store<T, TAIL>(static_cast<T*>(a.y) + (row0 + t) * a.d, k.col, a.d, y);
        }
    }
}

template <class T, int W, bool TAIL>
__global__ __launch_bounds__(256) void conv_bwd_kernel(const ConvArgs a) {
    const Walk k = walk_of(a);
    if (!k.on) return;
    Conv<T, W, TAIL> c;
    c.load(a, k.col);
    c.before(a, k.b, k.col, k.t0, k.len);
    float dw[W][4], db[4], dx[W][4];            // dx[j]: of the token j before the newest
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = dx[j][i] = 0.0f;
    }
    const int64_t row0 = (int64_t)k.b * a.length;
    const int end = k.t1 + W - 1;
    int since = W;                               // tokens since a sequence's start
    for (int t0 = k.t0; t0 < end; t0 += AHEAD) {
        Quad<T> q[AHEAD], r[AHEAD];
        bool start[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t row = row0 + max(min(t0 + i, a.length - 1), 0);
            if (a.length > 0) {
                q[i] = row_load<T, TAIL>(static_cast<const T*>(a.x) + row * a.x_stride, k.col, a.d);
                r[i] = row_load<T, TAIL>(static_cast<const T*>(a.dy) + row * a.dy_stride, k.col, a.d);
            } else {
                q[i] = r[i] = Quad<T>::zero();
            }
            start[i] = a.reset && t0 + i < k.len && a.reset[row] != 0;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int t = t0 + i;
            float v[4], g[4], p[4];
            take<TAIL>(q[i], k.col, a.d, v);
            take<TAIL>(r[i], k.col, a.d, g);
            const bool in = t < k.len;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = in ? v[e] : 0.0f;
            c.push(v, start[i]);
            c.sum(p);
            since = start[i] ? 0 : min(since + 1, W);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (a.act) {
                    const float s = sigmoid_of(p[e]);
                    g[e] *= s * (1.0f + p[e] * (1.0f - s));
                }
                g[e] = in ? g[e] : 0.0f;
                const float mine = t < k.t1 ? g[e] : 0.0f;  // of the tokens behind, dx alone is this piece's
                db[e] += mine;
#pragma unroll
                for (int j = 0; j < W; ++j) dw[W - 1 - j][e] = fmaf(mine, c.x[j][e], dw[W - 1 - j][e]);
#pragma unroll
                for (int j = W - 1; j >= 0; --j)
                    dx[j][e] = fmaf(c.w[W - 1 - j][e], since >= j ? g[e] : 0.0f, j ? dx[j - 1][e] : 0.0f);
            }
            // the token that no later one reaches
            const int done = t - (W - 1), late = done - (k.len - (W - 1));
            if (late >= 0 && late < W - 1 && a.dstate_out && done < a.length) {
                bool kept = true;                // its input is in the state that the row leaves
                for (int s = max(done + 1, 0); s < k.len; ++s) kept = kept && !(a.reset && a.reset[row0 + s] != 0);
                if (kept) {
                    float o[4];
                    take<TAIL>(row_load<T, TAIL>(static_cast<const T*>(a.dstate_out) + ((int64_t)k.b * (W - 1) + late) * a.d, k.col, a.d), k.col,
                               a.d, o);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dx[W - 1][e] += o[e];
                }
            }
            if (done >= k.t0 && done < k.t1) row_store<T, TAIL>(static_cast<T*>(a.dx) + (row0 + done) * a.d, k.col, a.d, dx[W - 1]);
            else if (done < 0 && k.piece == 0 && a.dstate)
                row_store<T, TAIL>(static_cast<T*>(a.dstate) + ((int64_t)k.b * (W - 1) + done + W - 1) * a.d, k.col, a.d, dx[W - 1]);
        }
    }
    float* part = a.part + ((int64_t)k.b * a.pieces + k.piece) * (W + 1) * a.d;
#pragma unroll
    for (int j = 0; j < W; ++j) row_store<float, TAIL>(part + (int64_t)j * a.d, k.col, a.d, dw[j]);
    row_store<float, TAIL>(part + (int64_t)W * a.d, k.col, a.d, db);
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
template <class T, int W, bool TAIL>
__global__ __launch_bounds__(256) void conv_step_kernel(const ConvArgs a) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, quads = (a.d + 3) / 4, b = x / quads;
    const int col = 4 * (int)(x % quads);
    if (b >= a.batch) return;
    Conv<T, W, TAIL> c;
    Quad<T> q[W];
    T* st = static_cast<T*>(const_cast<void*>(a.state)) + b * (W - 1) * a.d;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) q[k] = row_load<T, TAIL>(st + (int64_t)k * a.d, col, a.d);
    q[W - 1] = row_load<T, TAIL>(static_cast<const T*>(a.x) + b * a.x_stride, col, a.d);
    c.load(a, col);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        float v[4];
        take<TAIL>(q[k], col, a.d, v);
        c.push(v, false);
    }
    float y[4];
    c.sum(y);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (a.act) y[e] *= sigmoid_of(y[e]);
    row_store<T, TAIL>(static_cast<T*>(a.y) + b * a.d, col, a.d, y);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) row_store<T, TAIL>(st + (int64_t)k * a.d, col, a.d, c.x[W - 2 - k]);
}

enum Kind { FWD, BWD, STEP };
template <Kind K, class T, int W, bool TAIL>
void launch_one(const ConvArgs& a, hipStream_t s) {
    const int64_t threads = ceil_div(a.d, 4) * a.batch * (K == STEP ? 1 : a.pieces);
    const dim3 g((unsigned)ceil_div(threads, 256)), b(256);
    if (K == FWD) LRS_LAUNCH(K_CONV, (conv_fwd_kernel<T, W, TAIL>), g, b, 0, s, a);
    else if (K == BWD) LRS_LAUNCH(K_CONV_BWD, (conv_bwd_kernel<T, W, TAIL>), g, b, 0, s, a);
    else LRS_LAUNCH(K_CONV_STEP, (conv_step_kernel<T, W, TAIL>), g, b, 0, s, a);
}
template <Kind K, class T, int W>
void launch_tail(const ConvArgs& a, hipStream_t s) {
    if (a.d % 4) launch_one<K, T, W, true>(a, s);
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
