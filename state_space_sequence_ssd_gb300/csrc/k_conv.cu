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
// neighbouring channels and walks consecutive tokens with the last W-1 inputs in registers, a warp covers 32 V
// channels of a row, and a token's halo is read again only at the start of a thread's run of tokens, from L2.  Sums are float32; y, dx and the states are rounded once.
#include "ops.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 8;  // tokens of the forward kernel whose loads are in flight together
constexpr int kManyBlocks = 2 * kSms;  // two an SM: from there on a warp walks a long run of tokens

// The taps and biases of V channels as pairs.  Tap 3 is the current token's: a narrower kernel's taps end there and its
// first ones are unused (never multiplied: zero times an infinite input would be NaN).
template <int V>
__device__ __forceinline__ void load_taps(const float* __restrict__ weight, const float* __restrict__ bias, int W, int c,
                                          int valid, f32x2 (&w)[4][(V + 1) / 2], f32x2 (&b)[(V + 1) / 2]) {
    float wf[4][V + 1] = {}, bf[V + 1] = {};
    const bool rows = W == 4 && (reinterpret_cast<uintptr_t>(weight) & 15) == 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i >= valid) continue;
        if (rows) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(weight) + c + i);
            wf[0][i] = q.x; wf[1][i] = q.y; wf[2][i] = q.z; wf[3][i] = q.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k >= 4 - W) wf[k][i] = __ldg(weight + (int64_t)(c + i) * W + k - (4 - W));
        }
        if (bias != nullptr) bf[i] = __ldg(bias + c + i);
    }
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) {
        b[i] = pk(bf[2 * i], bf[2 * i + 1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k][i] = pk(wf[k][2 * i], wf[k][2 * i + 1]);
    }
}

// The convolution at one token: taps times the last four inputs (x[3] the newest), and the activation.
template <int W, int P>
__device__ __forceinline__ void taps_times(const f32x2 (&w)[4][P], const f32x2 (&b)[P], const f32x2 (*x)[P], f32x2 (&pre)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        pre[i] = b[i];
#pragma unroll
        for (int k = 4 - W; k < 4; ++k) pre[i] = fma2(w[k][i], x[k][i], pre[i]);
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
__device__ __forceinline__ Vec<T, V> input_at(const ConvArgs& a, int b, int t, int len, int c, int valid) {
    const Vec<T, V> z = Vec<T, V>::zero();
    if (t >= len) return z;
    if (t >= 0) return load_vec<T, V>(static_cast<const T*>(a.x) + b * a.x_batch + t * a.x_token + c, valid, true);
    if (a.init == nullptr || t < -(a.width - 1)) return z;
    return load_vec<T, V>(static_cast<const T*>(a.init) + ((int64_t)b * (a.width - 1) + t + a.width - 1) * a.channels + c,
                          valid, true);
}

// A warp: 32 V channels of RUN consecutive tokens, STEP of them loaded at a time, one step ahead of their use.  Runs whose
// tokens all count, most of them, are computed without looking at each.  Two channels a thread leave registers for 32 warps
// an SM: at 2 x 4096 x 4352 of bfloat16 29.7 us (4.8 TB/s; a plain copy of as many bytes takes 22.6), where four channels
// with half the warps take 33.3, steps of half as many tokens 33, runs of 16 tokens 34 and of 64 36.
template <typename T, int V, int W, int RUN>
__global__ void __launch_bounds__(32 * kWarps, 8) conv_forward_kernel(ConvArgs a, Pieces y, T* __restrict__ final_state) {
    constexpr int P = (V + 1) / 2, STEP = RUN < kStep ? RUN : kStep;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.z, c = (blockIdx.x * 32 + lane) * V;
    const int valid = min(V, a.channels - c);
    if (valid <= 0) return;
    const int len = row_length(a.lengths, b, a.seqlen);
    if (final_state != nullptr && blockIdx.y == 0 && warp < W - 1) {
        const Vec<T, V> v = input_at<T, V>(a, b, len - (W - 1) + warp, len, c, valid);
        store_vec<T, V>(final_state + ((int64_t)b * (W - 1) + warp) * a.channels + c, v, valid, true);
    }
    const int t0 = (blockIdx.y * kWarps + warp) * RUN;
    if (t0 >= a.seqlen) return;
    const int64_t xt = a.x_token;
    const T* xp = static_cast<const T*>(a.x) + b * a.x_batch + t0 * xt + c;
    const int wide = c < y.n[0] ? y.n[0] : c - y.n[0] < y.n[1] ? y.n[1] : y.n[2];
    T* yp = piece_at<T>(y, (int64_t)b * a.seqlen + t0, c);
    auto run = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        Vec<T, V> next[STEP];
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < STEP; ++i) {
                next[i] = load_vec<T, V>(xp, WHOLE || t + i < len ? valid : 0, true);
                xp += xt;
            }
        };
        fetch(t0);
        f32x2 x[STEP + 3][P];  // the inputs of this step's tokens, after the three before them
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const Vec<T, V> v = k >= 4 - W ? input_at<T, V>(a, b, t0 - 3 + k, len, c, valid) : Vec<T, V>::zero();
#pragma unroll
            for (int i = 0; i < P; ++i) x[k][i] = v.pair(i);
        }
        f32x2 w[4][P], bias[P];
        load_taps<V>(a.weight, a.bias, W, c, valid, w, bias);
#pragma unroll 1
        for (int s = 0; s < RUN; s += STEP) {
#pragma unroll
            for (int i = 0; i < STEP; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) x[3 + i][j] = next[i].pair(j);
            if (s + STEP < RUN) fetch(t0 + s + STEP);
#pragma unroll
            for (int i = 0; i < STEP; ++i) {
                const int t = t0 + s + i;
                f32x2 pre[P];
                taps_times<W, P>(w, bias, x + i, pre);
                if (a.silu) {
#pragma unroll
                    for (int j = 0; j < P; ++j) pre[j] = mul2(pre[j], sigmoid2(pre[j]));
                }
                store_vec<T, V>(yp, WHOLE || t < len ? Vec<T, V>::of_pairs(pre) : Vec<T, V>::zero(),
                                WHOLE || t < a.seqlen ? valid : 0, true);
                yp += wide;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) x[k][j] = x[STEP + k][j];
        }
    };
    if (t0 + RUN <= len) run(std::true_type());
    else run(std::false_type());
}

// The gradient's piece that holds channel c: its base, its width, the channel's place in it.
struct GradPiece {
    const void* p;
    int wide, at;
    bool f32;
};
__device__ __forceinline__ GradPiece grad_piece(const Pieces& dy, int c) {
    if (c < dy.n[0]) return {dy.p[0], dy.n[0], c, dy.f32[0] != 0};
    c -= dy.n[0];
    if (c < dy.n[1]) return {dy.p[1], dy.n[1], c, dy.f32[1] != 0};
    return {dy.p[2], dy.n[2], c - dy.n[1], dy.f32[2] != 0};
}

// A warp: 32 V channels of RUN consecutive tokens, their dx and their part of dweight and dbias.  dx[t] needs
// dLoss/dpre up to W-1 tokens on, so the walk goes that far past the run (those tokens' pre again).  Tokens are taken
// four at a time: their x and dy are loaded together, one group ahead of their use; groups whose tokens all count and
// all leave, most of them, are computed without looking at each.  The block's warps' sums of one channel are joined in
// shared memory in warp order and written as one row of `partial`, (rows, width + 1, channels).  Not bound by HBM (3.0 of
// 6.8 TB/s) nor by issue slots (58% used) but by latency: 18 warps an SM, which the registers allow, wait for each other's
// 13 multiply-adds, exponential and quotient per element and for loads.  At 2 x 4096 x 4352 of bfloat16 65 us, with the
// reduction, where 20 warps an SM hold two channels a thread; four channels and 12 warps 71, 16 warps 75, 24 warps 71,
// groups of two tokens 87 and of eight 82.
template <typename T, int V, int W, int RUN>
__global__ void __launch_bounds__(32 * kWarps, V == 2 ? 5 : 4) conv_backward_kernel(
    ConvArgs a, Pieces dy, const T* __restrict__ dfinal, T* __restrict__ dx, int64_t dx_batch, int64_t dx_token,
    T* __restrict__ dinit, float* __restrict__ partial) {
    constexpr int S = 4, P = (V + 1) / 2;
    __shared__ float sums[kWarps][W + 1][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.z, c = (blockIdx.x * 32 + lane) * V;
    constexpr int valid = V;  // channels are whole vectors
    const int len = row_length(a.lengths, b, a.seqlen);
    const int t0 = (blockIdx.y * kWarps + warp) * RUN;
    f32x2 dw[W][P], db[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        db[j] = 0ull;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][j] = 0ull;
    }
    if (c < a.channels && t0 < a.seqlen) {
        f32x2 w[4][P], bias[P];
        load_taps<V>(a.weight, a.bias, W, c, valid, w, bias);
        // the run itself; the first one also gives the initial state's tokens, which have no output of their own
        const int first = (t0 == 0 && dinit != nullptr) ? -(W - 1) : t0;
        const int last = min(t0 + RUN, a.seqlen), lim = min(len, last + W - 1);
        const GradPiece gr = grad_piece(dy, c);
        const int64_t gstep = (int64_t)gr.wide * (gr.f32 ? 4 : sizeof(T)), xstep = a.x_token;
        const char* gp = static_cast<const char*>(gr.p) + (((int64_t)b * a.seqlen + t0) * gr.wide + gr.at) * (gr.f32 ? 4 : sizeof(T));
        const T* xp = static_cast<const T*>(a.x) + b * a.x_batch + t0 * xstep + c;
        T* op = dx + b * dx_batch + (int64_t)(t0 - (W - 1)) * dx_token + c;  // of the token that leaves
        f32x2 x[S + 3][P], g[S + 3][P];  // inputs and dLoss/dpre of this group's tokens, after the three before them
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const Vec<T, V> v = k >= 4 - W ? input_at<T, V>(a, b, t0 - 3 + k, len, c, valid) : Vec<T, V>::zero();
#pragma unroll
            for (int j = 0; j < P; ++j) {
                x[k][j] = v.pair(j);
                g[k][j] = 0ull;
            }
        }
        Vec<T, V> nx[S];
        Vec<float, V> ng[S];  // dy as it lies in memory, in the first words where it is of 16 bits
        auto fetch = [&](int t) {
            auto load = [&](auto whole, auto wide) {
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    const int got = decltype(whole)::value || t + i < lim ? valid : 0;
                    nx[i] = load_vec<T, V>(xp, got, true);
                    xp += xstep;
                    if constexpr (decltype(wide)::value) {
                        ng[i] = load_vec<float, V>(reinterpret_cast<const float*>(gp), got, true);
                    } else {
                        const Vec<T, V> v = load_vec<T, V>(reinterpret_cast<const T*>(gp), got, true);
#pragma unroll
                        for (int u = 0; u < Vec<T, V>::WORDS; ++u) ng[i].w[u] = v.w[u];
                    }
                    gp += gstep;
                }
            };
            const bool all = t + S <= lim;
            if (sizeof(T) == 4 || gr.f32) all ? load(std::true_type(), std::true_type()) : load(std::false_type(), std::true_type());
            else all ? load(std::true_type(), std::false_type()) : load(std::false_type(), std::false_type());
        };
        // one group of tokens from t on; WHOLE: t + S <= min(len, last) and t - (W-1) >= first, no final state's gradient
        auto group = [&](int t, auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
            float pre[S][2 * P], gv[S][2 * P];
#pragma unroll
            for (int i = 0; i < S; ++i) {
                Vec<T, V> gt;
#pragma unroll
                for (int u = 0; u < Vec<T, V>::WORDS; ++u) gt.w[u] = ng[i].w[u];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    x[3 + i][j] = nx[i].pair(j);
                    f32x2 q = ng[i].pair(j);
                    if (sizeof(T) != 4 && !gr.f32) q = gt.pair(j);
                    unpk(q, gv[i][2 * j], gv[i][2 * j + 1]);
                }
            }
            if (t + S < last + W - 1) fetch(t + S);
#pragma unroll
            for (int i = 0; i < S; ++i) {
                f32x2 p[P];
                taps_times<W, P>(w, bias, x + i, p);
#pragma unroll
                for (int j = 0; j < P; ++j) unpk(p[j], pre[i][2 * j], pre[i][2 * j + 1]);
            }
            if (a.silu) {
#pragma unroll
                for (int i = 0; i < S; ++i)
#pragma unroll
                    for (int e = 0; e < 2 * P; ++e) {  // times s (1 + pre (1 - s))
                        const float s = sigmoid(pre[i][e]);
                        gv[i][e] *= fmaf(s * pre[i][e], 1.f - s, s);
                    }
            }
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    f32x2 q = pk(gv[i][2 * j], gv[i][2 * j + 1]);
                    if (!WHOLE && t + i >= len) q = 0ull;
                    g[3 + i][j] = q;
                    // the next run's tokens and those past the length add nothing, not zero times an infinite input
                    if (!WHOLE && t + i >= min(last, len)) continue;
                    db[j] = add2(db[j], q);
#pragma unroll
                    for (int k = 0; k < W; ++k) dw[k][j] = fma2(q, x[4 - W + k + i][j], dw[k][j]);
                }
            // the tokens W-1 before now have all their gradients and leave
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const int o = t + i - (W - 1);
                f32x2 d[P];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    d[j] = mul2(w[3][j], g[4 - W + i][j]);  // its own output's, through the newest tap
#pragma unroll
                    for (int k = 1; k < W; ++k) d[j] = fma2(w[3 - k][j], g[4 - W + k + i][j], d[j]);
                }
                if (WHOLE) {
                    store_vec<T, V>(op, Vec<T, V>::of_pairs(d), valid, true);
                } else if (o >= first && o < last) {
                    const int r = o + W - 1 - len;  // the final state's row that holds token o
                    if (dfinal != nullptr && r >= 0 && r < W - 1) {
                        const Vec<T, V> f = load_vec<T, V>(dfinal + ((int64_t)b * (W - 1) + r) * a.channels + c, valid, true);
#pragma unroll
                        for (int j = 0; j < P; ++j) d[j] = add2(d[j], f.pair(j));
                    }
                    store_vec<T, V>(o >= 0 ? op : dinit + ((int64_t)b * (W - 1) + o + W - 1) * a.channels + c,
                                    o < len ? Vec<T, V>::of_pairs(d) : Vec<T, V>::zero(), valid, true);
                }
                op += dx_token;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    x[k][j] = x[S + k][j];
                    g[k][j] = g[S + k][j];
                }
        };
        // tokens that leave before `calm` are no part of a final state
        const int calm = min(last, dfinal != nullptr ? len - (W - 1) : len);
        fetch(t0);
#pragma unroll 1
        for (int t = t0; t < last + W - 1; t += S) {
            if (t > t0 && t + S <= min(len, last) && t + S - (W - 1) <= calm) group(t, std::true_type());
            else group(t, std::false_type());
        }
    }
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float lo, hi;
            unpk(k < W ? dw[k < W ? k : 0][j] : db[j], lo, hi);
            sums[warp][k][lane * V + 2 * j] = lo;
            if (V > 1) sums[warp][k][lane * V + 2 * j + (V > 1)] = hi;
        }
    __syncthreads();
    const int64_t row = (int64_t)b * gridDim.y + blockIdx.y;
    for (int i = threadIdx.x; i < (W + 1) * 32 * V; i += blockDim.x) {
        const int k = i / (32 * V), cc = blockIdx.x * 32 * V + i % (32 * V);
        if (cc >= a.channels) continue;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) s += sums[q][k][i % (32 * V)];
        partial[(row * (W + 1) + k) * a.channels + cc] = s;
    }
}

// dweight (channels, W) and dbias from the rows of `partial`, summed in a fixed order: eight strided sums of
// rows, then those eight.
// (`partial` is written while this kernel may already run, so it is neither const for the kernel nor read as such.)
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float* partial, int rows, int channels, int W,
                                                          float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;  // (tap or bias, channel)
    const int n = (W + 1) * channels;
    grid_dep_wait();
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

// One token: a thread holds V channels of R rows, whose inputs it loads together; the taps are read once for them.  The
// slot's W-1 inputs are written back moved on by one.  An idle row (slot -1) writes zeros and leaves every slot alone.
template <typename T, int V, int W, int R>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs a, T* __restrict__ state, const int* __restrict__ slots,
                                                        int nslots, Pieces y, int* err) {
    constexpr int P = (V + 1) / 2;
    const int c = (blockIdx.x * blockDim.x + threadIdx.x) * V, b0 = blockIdx.y * R;
    const int valid = min(V, a.channels - c);
    if (valid <= 0) return;
    int slot[R];
    Vec<T, V> in[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) slot[r] = b0 + r < a.batch ? row_slot(slots, b0 + r, nslots, err) : -1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int got = slot[r] >= 0 ? valid : 0;
        const T* st = state + (int64_t)slot[r] * (W - 1) * a.channels + c;
        in[r][3] = load_vec<T, V>(static_cast<const T*>(a.x) + (b0 + r) * a.x_batch + c, got, true);
#pragma unroll
        for (int k = 4 - W; k < 3; ++k) in[r][k] = load_vec<T, V, true>(st + (int64_t)(k - (4 - W)) * a.channels, got, true);
    }
    f32x2 w[4][P], bias[P];
    load_taps<V>(a.weight, a.bias, W, c, valid, w, bias);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (b0 + r >= a.batch) return;
        Vec<T, V> out = Vec<T, V>::zero();
        if (slot[r] >= 0) {
            T* st = state + (int64_t)slot[r] * (W - 1) * a.channels + c;
#pragma unroll
            for (int k = 4 - W; k < 3; ++k) store_vec<T, V>(st + (int64_t)(k - (4 - W)) * a.channels, in[r][k + 1], valid, true);
            f32x2 x[4][P], pre[P];
#pragma unroll
            for (int k = 4 - W; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) x[k][j] = in[r][k].pair(j);
            taps_times<W, P>(w, bias, x, pre);
            if (a.silu) {
#pragma unroll
                for (int j = 0; j < P; ++j) pre[j] = mul2(pre[j], sigmoid2(pre[j]));
            }
            out = Vec<T, V>::of_pairs(pre);
        }
        store_vec<T, V>(piece_at<T>(y, b0 + r, c), out, valid, true);
    }
}

// Whether vectors of V elements of `size` bytes fit every row of the call: rows, strides and pieces are whole
// vectors from aligned bases.
bool whole_vectors(const ConvArgs& a, const Pieces& y, const void* s1, const void* s2, int V, int size) {
    const int bytes = V * size;
    if (a.channels % V || a.x_batch % V || a.x_token % V || !aligned_to(a.x, bytes) || !aligned_to(a.init, bytes) || !aligned_to(s1, bytes) ||
        !aligned_to(s2, bytes))
        return false;
    for (int i = 0; i < 3; ++i)
        if (y.n[i] % V || !aligned_to(y.p[i], y.f32[i] ? 4 * V : bytes)) return false;
    return true;
}

template <typename T, int V, int W>
void run_forward(const ConvArgs& a, const Pieces& y, void* final_state, cudaStream_t s) {
    const int tiles = ceil_div(a.channels, 32 * V);
    T* f = static_cast<T*>(final_state);
    // Long runs read the taps and the halo of W-1 tokens rarely; short ones fill the SMs on short prompts, and there only: the
    // grid of short runs holds kManyBlocks blocks of long ones at most.  (test_layer_sizes_gpu.py has the long runs.)
    constexpr int LONG = 32, SHORT = 4;
    static_assert(kManyBlocks * (LONG / SHORT) <= kMaxGrid, "short runs fit the grid");
    auto blocks = [&](int run) { return dim3(tiles, ceil_div(a.seqlen, kWarps * run), a.batch); };
    if ((int64_t)tiles * a.batch * ceil_div(a.seqlen, kWarps * LONG) >= kManyBlocks)
        conv_forward_kernel<T, V, W, LONG><<<blocks(LONG), 32 * kWarps, 0, s>>>(a, y, f);
    else
        conv_forward_kernel<T, V, W, SHORT><<<blocks(SHORT), 32 * kWarps, 0, s>>>(a, y, f);
}

template <typename T, int W>
int forward_of(const ConvArgs& a, const Pieces& y, void* final_state, cudaStream_t s) {
    launch_begin(kKindConv, s);
    if (whole_vectors(a, y, final_state, nullptr, 2, sizeof(T))) run_forward<T, 2, W>(a, y, final_state, s);
    else run_forward<T, 1, W>(a, y, final_state, s);
    return launch_end(kKindConv, s);
}

// Tokens that a warp of the backward kernel walks: long runs read the taps and the halo rarely and leave few rows of sums
// (at 2 x 4096 x 4352, an earlier form with runs of 16, 32 and 64 tokens: 110, 83 and 71 us), short ones fill the SMs where
// tokens are few.  (test_layer_sizes_gpu.py has the long runs.)
constexpr int kLongRun = 64, kShortRun = 16;
static_assert(kManyBlocks * (kLongRun / kShortRun) <= kMaxGrid, "short runs fit the grid");
int backward_run(const ConvArgs& a) {
    return (int64_t)a.batch * ceil_div(a.channels, 64) * ceil_div(a.seqlen, kWarps * kLongRun) >= kManyBlocks ? kLongRun : kShortRun;
}

template <typename T, int W>
int backward_of(const ConvArgs& a, const Pieces& dy, const void* dfinal, void* dx, int64_t dx_batch, int64_t dx_token,
                float* dweight, float* dbias, void* dinit, float* partial, cudaStream_t s) {
    const T* df = static_cast<const T*>(dfinal);
    T *o = static_cast<T*>(dx), *di = static_cast<T*>(dinit);
    const int run = backward_run(a), rows = ceil_div(a.seqlen, kWarps * run);
    const bool pairs = whole_vectors(a, dy, dfinal, dinit, 2, sizeof(T)) && dx_batch % 2 == 0 && dx_token % 2 == 0 &&
                       aligned_to(dx, 2 * sizeof(T));
    launch_begin(kKindConvBwd, s);
    auto go = [&](auto kernel, int channels) {
        kernel<<<dim3(ceil_div(a.channels, channels), rows, a.batch), 32 * kWarps, 0, s>>>(a, dy, df, o, dx_batch, dx_token, di,
                                                                                          partial);
    };
    if (pairs) {
        if (run == kLongRun) go(conv_backward_kernel<T, 2, W, kLongRun>, 64);
        else go(conv_backward_kernel<T, 2, W, kShortRun>, 64);
    } else {
        if (run == kLongRun) go(conv_backward_kernel<T, 1, W, kLongRun>, 32);
        else go(conv_backward_kernel<T, 1, W, kShortRun>, 32);
    }
    const int r = launch_end(kKindConvBwd, s);
    if (r != SSD_OK || (dweight == nullptr && dbias == nullptr)) return r;
    launch_begin(kKindConvBwd, s);
    launch_dependent(conv_reduce_kernel, dim3(ceil_div((a.width + 1) * a.channels, 32)), dim3(256), 0, s, partial, rows * a.batch,
                     a.channels, a.width, dweight, dbias);
    return launch_end(kKindConvBwd, s);
}

template <typename T, int V, int W>
void run_step(const ConvArgs& a, T* state, const int* slots, int nslots, const Pieces& y, int* err, cudaStream_t s) {
    const int tiles = ceil_div(a.channels, 128 * V);
    // four rows a thread where the batch fills the SMs all the same (test_layer_sizes_gpu.py has them)
    if (a.batch / 4 * tiles >= kSms)
        conv_step_kernel<T, V, W, 4><<<dim3(tiles, ceil_div(a.batch, 4)), 128, 0, s>>>(a, state, slots, nslots, y, err);
    else
        conv_step_kernel<T, V, W, 1><<<dim3(tiles, a.batch), 128, 0, s>>>(a, state, slots, nslots, y, err);
}

template <typename T, int W>
int step_of(const ConvArgs& a, void* state, const int* slots, int nslots, const Pieces& y, int* err, cudaStream_t s) {
    T* st = static_cast<T*>(state);
    launch_begin(kKindConvStep, s);
    if (whole_vectors(a, y, state, nullptr, 4, sizeof(T))) run_step<T, 4, W>(a, st, slots, nslots, y, err, s);
    else run_step<T, 1, W>(a, st, slots, nslots, y, err, s);
    return launch_end(kKindConvStep, s);
}

// Calls f with a value of the element type and the number of taps as a constant.
template <typename F>
int by_type_and_width(const ConvArgs& a, F f) {
    auto widths = [&](auto type) {
        if (a.width == 2) return f(type, std::integral_constant<int, 2>());
        if (a.width == 3) return f(type, std::integral_constant<int, 3>());
        return f(type, std::integral_constant<int, 4>());
    };
    if (a.dtype == SSD_BF16) return widths(__nv_bfloat16());
    if (a.dtype == SSD_F16) return widths(__half());
    return widths(0.f);
}

}  // namespace

int launch_conv_forward(const ConvArgs& a, const Pieces& y, void* final_state, cudaStream_t s) {
    return by_type_and_width(a, [&](auto type, auto W) { return forward_of<decltype(type), W()>(a, y, final_state, s); });
}

int conv_backward_rows(const ConvArgs& a) { return a.batch * ceil_div(a.seqlen, kWarps * backward_run(a)); }

int launch_conv_backward(const ConvArgs& a, const Pieces& dy, const void* dfinal, void* dx, int64_t dx_batch,
                         int64_t dx_token, float* dweight, float* dbias, void* dinit, float* partial, cudaStream_t s) {
    return by_type_and_width(a, [&](auto type, auto W) {
        return backward_of<decltype(type), W()>(a, dy, dfinal, dx, dx_batch, dx_token, dweight, dbias, dinit, partial, s);
    });
}

int launch_conv_step(const ConvArgs& a, void* state, const int* slots, int nslots, const Pieces& y, int* err,
                     cudaStream_t s) {
    return by_type_and_width(a, [&](auto type, auto W) { return step_of<decltype(type), W()>(a, state, slots, nslots, y, err, s); });
}

}  // namespace ssd
