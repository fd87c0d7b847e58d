// k_conv.cu -- the short causal depthwise convolution in front of a scan, its gradient, and its step for
// single tokens.  Per row b, channel c and token t, with W = width taps:
//
//   pre[t] = bias[c] + sum_k weight[c][k] x[t - (W-1) + k],   y[t] = pre[t] sigmoid(pre[t])  (or pre[t])
//
// where x at negative t is the initial state (the W-1 inputs before the row, zeros without one), and the
// final state is the last W-1 inputs of the row's own length.  With g = dLoss/dpre:
//
//   dx[t] = sum_k weight[c][k] g[t + (W-1) - k] + (dfinal where t is one of the last W-1 tokens),
//   dweight[c][k] = sum_{b,t} g[t] x[t - (W-1) + k],   dbias[c] = sum_{b,t} g[t].
//
// Every kernel is bound by HBM: the inputs are read once, the outputs written once, and a handful of
// multiply-adds with one exponential and one quotient per element hide under that.  So a thread holds V
// neighbouring channels (16 bytes in the forward pass) and walks consecutive tokens with the last W-1 inputs
// in registers, a warp covers 32 V channels of a row, and a token's halo is read again only at the start of
// a thread's run of tokens, from L2.  Sums are float32; y, dx and the states are rounded once.
#include "ops.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;

template <int V>
__device__ __forceinline__ void load_taps(const float* __restrict__ weight, const float* __restrict__ bias, int W, int c,
                                          int valid, float (&w)[4][V], float (&b)[V]) {
    // tap 3 is the current token's: a narrower kernel's taps end there and its first ones are unused (never
    // multiplied: zero times an infinite input would be NaN)
#pragma unroll
    for (int i = 0; i < V; ++i) {
        b[i] = (bias != nullptr && i < valid) ? bias[c + i] : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k][i] = (k >= 4 - W && i < valid) ? weight[(int64_t)(c + i) * W + k - (4 - W)] : 0.f;
    }
}

// Where channel c's piece starts, and its row of (batch * seqlen) row `row`.
template <typename T>
__device__ __forceinline__ T* piece_at(const Pieces& y, int64_t row, int c) {
    if (c < y.n[0]) return static_cast<T*>(y.p[0]) + row * y.n[0] + c;
    c -= y.n[0];
    if (c < y.n[1]) return static_cast<T*>(y.p[1]) + row * y.n[1] + c;
    return static_cast<T*>(y.p[2]) + row * y.n[2] + (c - y.n[1]);
}

// x at token t of row b (t < 0: the initial state's rows; past the length: zero)
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> input_at(const ConvArgs& a, int b, int t, int len, int c, int valid, bool vec) {
    Vec<T, V> z;
#pragma unroll
    for (int i = 0; i < V; ++i) z.e[i] = from_f32<T>(0.f);
    if (t >= len) return z;
    if (t >= 0) return load_vec<T, V>(static_cast<const T*>(a.x) + b * a.x_batch + t * a.x_token + c, valid, vec);
    if (a.init == nullptr || t < -(a.width - 1)) return z;
    return load_vec<T, V>(static_cast<const T*>(a.init) + ((int64_t)b * (a.width - 1) + t + a.width - 1) * a.channels + c,
                          valid, vec);
}

// A warp: 32 V channels of `run` consecutive tokens.
template <typename T, int V, int RUN>
__global__ void __launch_bounds__(32 * kWarps) conv_forward_kernel(ConvArgs a, Pieces y, T* __restrict__ final_state,
                                                                   bool vec) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.z, c = (blockIdx.x * 32 + lane) * V;
    const int valid = min(V, a.channels - c);
    if (valid <= 0) return;
    const int len = row_length(a.lengths, b, a.seqlen);
    const int64_t row0 = (int64_t)b * a.seqlen;
    if (final_state != nullptr && blockIdx.y == 0 && warp < a.width - 1) {
        const Vec<T, V> v = input_at<T, V>(a, b, len - (a.width - 1) + warp, len, c, valid, vec);
        store_vec<T, V>(final_state + ((int64_t)b * (a.width - 1) + warp) * a.channels + c, v, valid, vec);
    }
    const int t0 = (blockIdx.y * kWarps + warp) * RUN;
    if (t0 >= a.seqlen) return;
    float w[4][V], bias[V];
    load_taps<V>(a.weight, a.bias, a.width, c, valid, w, bias);
    Vec<T, V> past[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) past[k] = input_at<T, V>(a, b, t0 - 3 + k, len, c, valid, vec);
    constexpr int STEP = RUN < 8 ? RUN : 8;  // tokens whose loads are in flight together
#pragma unroll 1
    for (int s = 0; s < RUN; s += STEP) {
        Vec<T, V> in[STEP + 3];
#pragma unroll
        for (int k = 0; k < 3; ++k) in[k] = past[k];
#pragma unroll
        for (int i = 0; i < STEP; ++i) in[3 + i] = input_at<T, V>(a, b, t0 + s + i, len, c, valid, vec);
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
            const int t = t0 + s + i;
            if (t >= a.seqlen) return;
            Vec<T, V> out;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float v = bias[e];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k >= 4 - a.width) v = fmaf(w[k][e], to_f32<T>(in[i + k].e[e]), v);
                if (a.silu) v *= sigmoid(v);
                out.e[e] = from_f32<T>(t < len ? v : 0.f);
            }
            store_vec<T, V>(piece_at<T>(y, row0 + t, c), out, valid, vec);
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) past[k] = in[STEP + k];
    }
}

// dLoss/dpre at token t from dLoss/dy and pre
__device__ __forceinline__ float through_silu(float dy, float pre, int silu) {
    if (!silu) return dy;
    const float s = sigmoid(pre);
    return dy * s * fmaf(pre, 1.f - s, 1.f);
}

template <typename T, int V>
__device__ __forceinline__ void grad_at(const Pieces& dy, int64_t row, int c, int valid, bool vec, float (&g)[V]) {
    int p = 0, at = c;
    if (at >= dy.n[0]) { at -= dy.n[0]; p = 1; if (at >= dy.n[1]) { at -= dy.n[1]; p = 2; } }
    const void* base = p == 0 ? dy.p[0] : p == 1 ? dy.p[1] : dy.p[2];
    const int n = p == 0 ? dy.n[0] : p == 1 ? dy.n[1] : dy.n[2];
    const int f32 = p == 0 ? dy.f32[0] : p == 1 ? dy.f32[1] : dy.f32[2];
    if (f32) {
        const Vec<float, V> r = load_vec<float, V>(static_cast<const float*>(base) + row * n + at, valid, vec);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = r.e[i];
    } else {
        const Vec<T, V> r = load_vec<T, V>(static_cast<const T*>(base) + row * n + at, valid, vec);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = to_f32<T>(r.e[i]);
    }
}

constexpr int kBwdRun = 32;  // tokens a warp of the backward kernel walks

// A warp: 32 V channels of kBwdRun consecutive tokens, their dx and their part of dweight and dbias.  dx[t]
// needs dLoss/dpre up to W-1 tokens on, so the walk goes that far past the run (those tokens' pre again).
// The block's eight warps' sums of one channel are joined in shared memory in warp order and written as one
// row of `partial`, (rows, width + 1, channels).
template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps) conv_backward_kernel(ConvArgs a, Pieces dy, const T* __restrict__ dfinal,
                                                                    T* __restrict__ dx, int64_t dx_batch, int64_t dx_token,
                                                                    T* __restrict__ dinit, float* __restrict__ partial,
                                                                    bool vec, bool vec_dx) {
    __shared__ float sums[kWarps][5][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.z, c = (blockIdx.x * 32 + lane) * V, W = a.width;
    const int valid = max(0, min(V, a.channels - c));
    const int len = row_length(a.lengths, b, a.seqlen);
    const int64_t row0 = (int64_t)b * a.seqlen;
    const int t0 = (blockIdx.y * kWarps + warp) * kBwdRun;
    float w[4][V], bias[V], dw[4][V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) dw[k][e] = 0.f;
    }
    if (valid > 0) load_taps<V>(a.weight, a.bias, W, c, valid, w, bias);
    if (valid > 0 && t0 < a.seqlen) {
        // the run itself; block row 0 also walks the initial state's tokens, which have no output of their own
        const int first = (t0 == 0 && dinit != nullptr) ? -(W - 1) : t0;
        const int last = min(t0 + kBwdRun, a.seqlen);
        float x[4][V], g[4][V];  // the last four inputs and dLoss/dpre values, newest at [3]
#pragma unroll
        for (int e = 0; e < V; ++e)
#pragma unroll
            for (int k = 0; k < 4; ++k) g[k][e] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const Vec<T, V> r = input_at<T, V>(a, b, t0 - 4 + k, len, c, valid, vec);
#pragma unroll
            for (int e = 0; e < V; ++e) x[k][e] = to_f32<T>(r.e[e]);
        }
#pragma unroll 4
        for (int t = t0; t < last + W - 1; ++t) {
            // token t enters; token t - (W-1) has all its gradients and leaves
            const Vec<T, V> r = input_at<T, V>(a, b, t, len, c, valid, vec);
            float gy[V];
            const bool live = t < len;
            if (live) grad_at<T, V>(dy, row0 + t, c, valid, vec, gy);
#pragma unroll
            for (int e = 0; e < V; ++e) {
#pragma unroll
                for (int k = 0; k < 3; ++k) { x[k][e] = x[k + 1][e]; g[k][e] = g[k + 1][e]; }
                x[3][e] = to_f32<T>(r.e[e]);
                float pre = bias[e];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k >= 4 - W) pre = fmaf(w[k][e], x[k][e], pre);
                g[3][e] = live ? through_silu(gy[e], pre, a.silu) : 0.f;
                if (t < last) {
                    db[e] += g[3][e];
#pragma unroll
                    for (int k = 0; k < 4; ++k) dw[k][e] = fmaf(g[3][e], x[k][e], dw[k][e]);
                }
            }
            const int o = t - (W - 1);
            if (o < first || o >= last) continue;
            // g[3] is token t's: tap 3 - j of token o's own later outputs, at distance j
            float d[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                d[e] = 0.f;
                if (W == 4) d[e] = w[3][e] * g[0][e] + w[2][e] * g[1][e] + w[1][e] * g[2][e] + w[0][e] * g[3][e];
                else if (W == 3) d[e] = w[3][e] * g[1][e] + w[2][e] * g[2][e] + w[1][e] * g[3][e];
                else d[e] = w[3][e] * g[2][e] + w[2][e] * g[3][e];
            }
            const int j = o + W - 1 - len;  // the final state's row that holds token o
            if (dfinal != nullptr && j >= 0 && j < W - 1) {
                const Vec<T, V> f = load_vec<T, V>(dfinal + ((int64_t)b * (W - 1) + j) * a.channels + c, valid, vec);
#pragma unroll
                for (int e = 0; e < V; ++e) d[e] += to_f32<T>(f.e[e]);
            }
            Vec<T, V> out;
#pragma unroll
            for (int e = 0; e < V; ++e) out.e[e] = from_f32<T>((o < len) ? d[e] : 0.f);
            if (o >= 0)
                store_vec<T, V>(dx + b * dx_batch + o * dx_token + c, out, valid, vec_dx);
            else
                store_vec<T, V>(dinit + ((int64_t)b * (W - 1) + o + W - 1) * a.channels + c, out, valid, vec);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < 4; ++k) sums[warp][k][lane * V + e] = dw[k][e];
        sums[warp][4][lane * V + e] = db[e];
    }
    __syncthreads();
    const int64_t row = (int64_t)b * gridDim.y + blockIdx.y;
    for (int i = threadIdx.x; i < 5 * 32 * V; i += blockDim.x) {
        const int k = i / (32 * V), cc = blockIdx.x * 32 * V + i % (32 * V);
        if (cc >= a.channels || k < 4 - W) continue;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) s += sums[q][k][i % (32 * V)];
        partial[(row * (W + 1) + k - (4 - W)) * a.channels + cc] = s;
    }
}

// dweight (channels, W) and dbias from the rows of `partial`, summed in a fixed order: eight strided sums of
// rows, then those eight.
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float* __restrict__ partial, int rows, int channels, int W,
                                                          float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;  // (tap or bias, channel)
    const int n = (W + 1) * channels;
    float s = 0.f;
    if (i < n) {
#pragma unroll 8
        for (int r = warp; r < rows; r += 8) s += partial[(int64_t)r * n + i];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || i >= n) return;
    s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += part[q][lane];
    const int k = i / channels, c = i % channels;
    if (k < W) {
        if (dweight != nullptr) dweight[(int64_t)c * W + k] = s;
    } else if (dbias != nullptr) {
        dbias[c] = s;
    }
}

// One token: a thread holds V channels of one row, reads the slot's W-1 inputs, and writes them back moved on
// by one.  An idle row (slot -1) writes zeros and leaves every slot alone.
template <typename T, int V>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs a, T* __restrict__ state, const int* __restrict__ slots,
                                                        int nslots, Pieces y, int* err, bool vec) {
    const int c = (blockIdx.x * blockDim.x + threadIdx.x) * V, b = blockIdx.y;
    const int valid = min(V, a.channels - c);
    if (valid <= 0) return;
    const int W = a.width, slot = row_slot(slots, b, nslots, err);
    Vec<T, V> out;
#pragma unroll
    for (int e = 0; e < V; ++e) out.e[e] = from_f32<T>(0.f);
    if (slot >= 0) {
        T* st = state + (int64_t)slot * (W - 1) * a.channels + c;
        Vec<T, V> in[4];
        in[3] = load_vec<T, V>(static_cast<const T*>(a.x) + b * a.x_batch + c, valid, vec);
#pragma unroll
        for (int k = 0; k < 3; ++k)
            in[k] = k >= 4 - W ? load_vec<T, V>(st + (int64_t)(k - (4 - W)) * a.channels, valid, vec) : out;
        float w[4][V], bias[V];
        load_taps<V>(a.weight, a.bias, W, c, valid, w, bias);
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k >= 4 - W) store_vec<T, V>(st + (int64_t)(k - (4 - W)) * a.channels, in[k + 1], valid, vec);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float v = bias[e];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k >= 4 - W) v = fmaf(w[k][e], to_f32<T>(in[k].e[e]), v);
            if (a.silu) v *= sigmoid(v);
            out.e[e] = from_f32<T>(v);
        }
    }
    store_vec<T, V>(piece_at<T>(y, b, c), out, valid, vec);
}

bool on(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Whether vectors of V elements of `size` bytes fit every row of the call: rows, strides and pieces are whole
// vectors from aligned bases.
bool whole_vectors(const ConvArgs& a, const Pieces& y, const void* s1, const void* s2, int V, int size) {
    const int bytes = V * size;
    if (a.channels % V || a.x_batch % V || a.x_token % V || !on(a.x, bytes) || !on(a.init, bytes) || !on(s1, bytes) ||
        !on(s2, bytes))
        return false;
    for (int i = 0; i < 3; ++i)
        if (y.n[i] % V || !on(y.p[i], y.f32[i] ? 4 * V : bytes)) return false;
    return true;
}

template <typename T, int V>
void run_forward(const ConvArgs& a, const Pieces& y, void* final_state, bool vec, cudaStream_t s) {
    const int tiles = ceil_div(a.channels, 32 * V);
    // long runs read the halo of W-1 tokens rarely; short ones fill the SMs on short prompts
    const bool many = (int64_t)tiles * a.batch * ceil_div(a.seqlen, kWarps * 16) >= 304;
    if (many)
        conv_forward_kernel<T, V, 16><<<dim3(tiles, ceil_div(a.seqlen, kWarps * 16), a.batch), 32 * kWarps, 0, s>>>(
            a, y, static_cast<T*>(final_state), vec);
    else
        conv_forward_kernel<T, V, 4><<<dim3(tiles, ceil_div(a.seqlen, kWarps * 4), a.batch), 32 * kWarps, 0, s>>>(
            a, y, static_cast<T*>(final_state), vec);
}

template <typename T>
int forward_of(const ConvArgs& a, const Pieces& y, void* final_state, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    launch_begin(kKindConv, s);
    if (whole_vectors(a, y, final_state, nullptr, V, sizeof(T))) run_forward<T, V>(a, y, final_state, true, s);
    else run_forward<T, 1>(a, y, final_state, true, s);
    return launch_end(kKindConv, s);
}

template <typename T>
int backward_of(const ConvArgs& a, const Pieces& dy, const void* dfinal, void* dx, int64_t dx_batch, int64_t dx_token,
                float* dweight, float* dbias, void* dinit, float* partial, cudaStream_t s) {
    constexpr int V = 4;
    const T* df = static_cast<const T*>(dfinal);
    T *o = static_cast<T*>(dx), *di = static_cast<T*>(dinit);
    const int rows = ceil_div(a.seqlen, kWarps * kBwdRun);
    launch_begin(kKindConvBwd, s);
    if (whole_vectors(a, dy, dfinal, dinit, V, sizeof(T))) {
        const bool vec_dx = dx_batch % V == 0 && dx_token % V == 0 && on(dx, V * sizeof(T));
        conv_backward_kernel<T, V><<<dim3(ceil_div(a.channels, 32 * V), rows, a.batch), 32 * kWarps, 0, s>>>(
            a, dy, df, o, dx_batch, dx_token, di, partial, true, vec_dx);
    } else {
        conv_backward_kernel<T, 1><<<dim3(ceil_div(a.channels, 32), rows, a.batch), 32 * kWarps, 0, s>>>(
            a, dy, df, o, dx_batch, dx_token, di, partial, true, true);
    }
    const int r = launch_end(kKindConvBwd, s);
    if (r != SSD_OK || (dweight == nullptr && dbias == nullptr)) return r;
    launch_begin(kKindConvBwd, s);
    conv_reduce_kernel<<<ceil_div((a.width + 1) * a.channels, 32), 256, 0, s>>>(partial, rows * a.batch, a.channels, a.width,
                                                                               dweight, dbias);
    return launch_end(kKindConvBwd, s);
}

template <typename T>
int step_of(const ConvArgs& a, void* state, const int* slots, int nslots, const Pieces& y, int* err, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    launch_begin(kKindConvStep, s);
    if (whole_vectors(a, y, state, nullptr, V, sizeof(T)))
        conv_step_kernel<T, V><<<dim3(ceil_div(a.channels, 128 * V), a.batch), 128, 0, s>>>(a, static_cast<T*>(state), slots,
                                                                                         nslots, y, err, true);
    else
        conv_step_kernel<T, 1><<<dim3(ceil_div(a.channels, 128), a.batch), 128, 0, s>>>(a, static_cast<T*>(state), slots,
                                                                                       nslots, y, err, true);
    return launch_end(kKindConvStep, s);
}

}  // namespace

int launch_conv_forward(const ConvArgs& a, const Pieces& y, void* final_state, cudaStream_t s) {
    if (a.dtype == SSD_BF16) return forward_of<__nv_bfloat16>(a, y, final_state, s);
    if (a.dtype == SSD_F16) return forward_of<__half>(a, y, final_state, s);
    return forward_of<float>(a, y, final_state, s);
}

int conv_backward_rows(const ConvArgs& a) { return a.batch * ceil_div(a.seqlen, kWarps * kBwdRun); }

int launch_conv_backward(const ConvArgs& a, const Pieces& dy, const void* dfinal, void* dx, int64_t dx_batch,
                         int64_t dx_token, float* dweight, float* dbias, void* dinit, float* partial, cudaStream_t s) {
    if (a.dtype == SSD_BF16)
        return backward_of<__nv_bfloat16>(a, dy, dfinal, dx, dx_batch, dx_token, dweight, dbias, dinit, partial, s);
    if (a.dtype == SSD_F16)
        return backward_of<__half>(a, dy, dfinal, dx, dx_batch, dx_token, dweight, dbias, dinit, partial, s);
    return backward_of<float>(a, dy, dfinal, dx, dx_batch, dx_token, dweight, dbias, dinit, partial, s);
}

int launch_conv_step(const ConvArgs& a, void* state, const int* slots, int nslots, const Pieces& y, int* err,
                     cudaStream_t s) {
    if (a.dtype == SSD_BF16) return step_of<__nv_bfloat16>(a, state, slots, nslots, y, err, s);
    if (a.dtype == SSD_F16) return step_of<__half>(a, state, slots, nslots, y, err, s);
    return step_of<float>(a, state, slots, nslots, y, err, s);
}

}  // namespace ssd
