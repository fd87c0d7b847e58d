// k_norm.cu -- layer norm over the last dimension, and its gradient with the weight's and the bias's.
//
//   xhat = (x - mean) rstd,   y = xhat weight + bias,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   dx = rstd (gw - mean(gw) - xhat mean(gw xhat)),  gw = dy weight
//   dweight = sum over rows of dy xhat,   dbias = sum over rows of dy
//
// Bound by HBM: a row is read once and held in registers (mean first, then the squares around it: no
// cancellation of large sums), and written once.  `lanes` threads share a row, a power of two of at most a
// block's; narrow rows share a block.  The backward kernel's blocks each walk rows a grid's width apart and
// hold the columns' sums of their threads in registers; a block writes one row of partial sums and a second
// kernel adds the blocks' rows in a fixed order.  All sums are float32; y and dx are rounded once.
#include "ops.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;

// Sum over the `lanes` threads of one row (a power of two; at most kThreads).  Every thread of the block calls it.
// `lane` is the thread's place in its row; buf holds one float per warp.
__device__ __forceinline__ float row_sum(float v, int lanes, float* buf) {
    for (int o = min(lanes, 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lanes <= 32) return v;
    const int warp = threadIdx.x >> 5, per = lanes >> 5;
    __syncthreads();  // buf's last readers are done
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < per; ++i) v += buf[(warp / per) * per + i];
    return v;
}

// NV vectors of V columns per thread: thread `lane` holds columns (lane + lanes i) V ..  With NV = 0 the row
// does not fit the registers and is read again (from L2) for each sum.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const T* __restrict__ x, int64_t x_row,
                                                                const float* __restrict__ weight,
                                                                const float* __restrict__ bias, float eps, int64_t rows,
                                                                int width, int lanes, T* __restrict__ y,
                                                                float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float buf[kThreads / 32];
    const int lane = threadIdx.x % lanes;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    const bool live = row < rows;
    const T* xr = x + (live ? row : 0) * x_row;
    const float inv = 1.f / (float)width;
    float v[NV > 0 ? NV : 1][V];
    float s = 0.f;
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + lanes * i) * V;
            const Vec<T, V> r = load_vec<T, V>(xr + c, live ? width - c : 0, true);
#pragma unroll
            for (int e = 0; e < V; ++e) { v[i][e] = to_f32<T>(r.e[e]); s += v[i][e]; }
        }
    } else if (live) {
        for (int c = lane; c < width; c += lanes) s += to_f32<T>(xr[c]);
    }
    const float m = row_sum(s, lanes, buf) * inv;
    float q = 0.f;
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e)
                if ((lane + lanes * i) * V + e < width) { v[i][e] -= m; q = fmaf(v[i][e], v[i][e], q); }
    } else if (live) {
        for (int c = lane; c < width; c += lanes) { const float d = to_f32<T>(xr[c]) - m; q = fmaf(d, d, q); }
    }
    const float rs = rsqrtf(fmaf(row_sum(q, lanes, buf), inv, eps));
    if (!live) return;
    if (lane == 0) {
        if (mean != nullptr) mean[row] = m;
        if (rstd != nullptr) rstd[row] = rs;
    }
    T* yr = y + row * width;
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + lanes * i) * V;
            if (c >= width) break;
            Vec<T, V> o;
            const Vec<float, V> w = weight != nullptr ? load_vec<float, V>(weight + c, width - c, false) : Vec<float, V>();
            const Vec<float, V> bb = bias != nullptr ? load_vec<float, V>(bias + c, width - c, false) : Vec<float, V>();
#pragma unroll
            for (int e = 0; e < V; ++e)
                o.e[e] = from_f32<T>(fmaf(v[i][e] * rs, weight != nullptr ? w.e[e] : 1.f, bias != nullptr ? bb.e[e] : 0.f));
            store_vec<T, V>(yr + c, o, width - c, true);
        }
    } else {
        for (int c = lane; c < width; c += lanes)
            yr[c] = from_f32<T>(fmaf((to_f32<T>(xr[c]) - m) * rs, weight != nullptr ? weight[c] : 1.f,
                                     bias != nullptr ? bias[c] : 0.f));
    }
}

// A block of `lanes` threads a row, kThreads / lanes rows at a time.  The thread's columns of dweight and dbias
// stay in registers while the block walks its rows.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const T* __restrict__ x, int64_t x_row,
                                                                 const float* __restrict__ weight,
                                                                 const float* __restrict__ mean,
                                                                 const float* __restrict__ rstd, const T* __restrict__ dy,
                                                                 int64_t dy_row, int64_t rows, int width, int lanes,
                                                                 T* __restrict__ dx, float* __restrict__ partial) {
    extern __shared__ float sums[];  // (kThreads / lanes) x 2 x width where rows share a block
    __shared__ float buf[2][kThreads / 32];
    const int lane = threadIdx.x % lanes, slot = threadIdx.x / lanes, per = kThreads / lanes;
    const float inv = 1.f / (float)width;
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = (lane + lanes * i) * V + e;
            w[i][e] = c < width ? (weight != nullptr ? weight[c] : 1.f) : 0.f;
            dw[i][e] = db[i][e] = 0.f;
        }
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < rows; r0 += (int64_t)gridDim.x * per) {
        const int64_t row = r0 + slot;
        const bool live = row < rows;
        const T* xr = x + (live ? row : 0) * x_row;
        const T* gr = dy + (live ? row : 0) * dy_row;
        const float m = live ? mean[row] : 0.f, rs = live ? rstd[row] : 0.f;
        float xh[NV][V], g[NV][V];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + lanes * i) * V;
            const Vec<T, V> a = load_vec<T, V>(xr + c, live ? width - c : 0, true);
            const Vec<T, V> d = load_vec<T, V>(gr + c, live ? width - c : 0, true);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float gy = to_f32<T>(d.e[e]);
                xh[i][e] = (live && c + e < width) ? (to_f32<T>(a.e[e]) - m) * rs : 0.f;
                db[i][e] += gy;
                dw[i][e] = fmaf(gy, xh[i][e], dw[i][e]);
                g[i][e] = gy * w[i][e];
                s1 += g[i][e];
                s2 = fmaf(g[i][e], xh[i][e], s2);
            }
        }
        s1 = row_sum(s1, lanes, buf[0]) * inv;
        s2 = row_sum(s2, lanes, buf[1]) * inv;
        if (!live) continue;
        T* o = dx + row * width;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + lanes * i) * V;
            if (c >= width) break;
            Vec<T, V> out;
#pragma unroll
            for (int e = 0; e < V; ++e) out.e[e] = from_f32<T>(rs * (g[i][e] - s1 - xh[i][e] * s2));
            store_vec<T, V>(o + c, out, width - c, true);
        }
    }
    if (partial == nullptr) return;
    float* row = partial + (int64_t)blockIdx.x * 2 * width;
    if (per == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int c = (lane + lanes * i) * V + e;
                if (c < width) { row[c] = dw[i][e]; row[width + c] = db[i][e]; }
            }
        return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = (lane + lanes * i) * V + e;
            if (c < width) { sums[slot * 2 * width + c] = dw[i][e]; sums[slot * 2 * width + width + c] = db[i][e]; }
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * width; c += kThreads) {
        float s = 0.f;
        for (int q = 0; q < per; ++q) s += sums[q * 2 * width + c];
        row[c] = s;
    }
}

// Rows wider than the registers hold: a block per row at a time, x and dy read twice (the second time from L2),
// the columns' sums kept in the block's row of `partial`.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_wide_kernel(const T* __restrict__ x, int64_t x_row,
                                                                      const float* __restrict__ weight,
                                                                      const float* __restrict__ mean,
                                                                      const float* __restrict__ rstd,
                                                                      const T* __restrict__ dy, int64_t dy_row,
                                                                      int64_t rows, int width, T* __restrict__ dx,
                                                                      float* __restrict__ partial) {
    __shared__ float buf[2][kThreads / 32];
    const float inv = 1.f / (float)width;
    float* sum = partial == nullptr ? nullptr : partial + (int64_t)blockIdx.x * 2 * width;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T *xr = x + row * x_row, *gr = dy + row * dy_row;
        const float m = mean[row], rs = rstd[row];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float gy = to_f32<T>(gr[c]), xh = (to_f32<T>(xr[c]) - m) * rs;
            const float g = gy * (weight != nullptr ? weight[c] : 1.f);
            if (sum != nullptr) {
                const bool first = row == blockIdx.x;
                sum[c] = first ? gy * xh : fmaf(gy, xh, sum[c]);
                sum[width + c] = first ? gy : sum[width + c] + gy;
            }
            s1 += g;
            s2 = fmaf(g, xh, s2);
        }
        s1 = row_sum(s1, kThreads, buf[0]) * inv;
        s2 = row_sum(s2, kThreads, buf[1]) * inv;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float g = to_f32<T>(gr[c]) * (weight != nullptr ? weight[c] : 1.f), xh = (to_f32<T>(xr[c]) - m) * rs;
            dx[row * width + c] = from_f32<T>(rs * (g - s1 - xh * s2));
        }
    }
}

// dweight and dbias from the blocks' rows of `partial`: eight strided sums, then those eight.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* __restrict__ partial, int parts, int width,
                                                          float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (i < 2 * width) {
#pragma unroll 8
        for (int r = warp; r < parts; r += 8) s += partial[(int64_t)r * 2 * width + i];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || i >= 2 * width) return;
    s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += part[q][lane];
    if (i < width) {
        if (dweight != nullptr) dweight[i] = s;
    } else if (dbias != nullptr) {
        dbias[i - width] = s;
    }
}

bool on(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Threads that share a row of `vecs` vectors, a power of two: one vector each up to a warp, then up to a block's
// threads so that a thread holds about `want` vectors.
int row_lanes(int vecs, int want) {
    int lanes = 1;
    while (lanes < 32 && lanes < vecs) lanes *= 2;
    while (lanes < kThreads && lanes * want < vecs) lanes *= 2;
    return lanes;
}

template <typename T, int V>
int forward_of(const void* x, int64_t x_row, const float* weight, const float* bias, float eps, int64_t rows, int width,
               void* y, float* mean, float* rstd, cudaStream_t s) {
    const int vecs = ceil_div(width, V);
    const int lanes = row_lanes(vecs, V == 1 ? 8 : 2);
    const int nv = ceil_div(vecs, lanes);
    const int64_t blocks = ceil_div64(rows, kThreads / lanes);
    if (blocks > 2147483647) return SSD_ERR_UNSUPPORTED;
    launch_begin(kKindNorm, s);
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)blocks, kThreads, 0, s>>>(static_cast<const T*>(x), x_row, weight, bias, eps, rows, width, lanes,
                                                     static_cast<T*>(y), mean, rstd);
    };
    constexpr int M = V == 1 ? 4 : 1;
    if (nv <= 1 * M) go(norm_forward_kernel<T, V, 1 * M>);
    else if (nv <= 2 * M) go(norm_forward_kernel<T, V, 2 * M>);
    else if (nv <= 4 * M) go(norm_forward_kernel<T, V, 4 * M>);
    else if (nv <= 8 * M) go(norm_forward_kernel<T, V, 8 * M>);
    else go(norm_forward_kernel<T, 1, 0>);
    return launch_end(kKindNorm, s);
}

template <typename T, int V>
int backward_of(const void* x, int64_t x_row, const float* weight, const float* mean, const float* rstd, const void* dy,
                int64_t dy_row, int64_t rows, int width, void* dx, float* partial, int parts, cudaStream_t s) {
    const int vecs = ceil_div(width, V);
    const int lanes = row_lanes(vecs, V == 1 ? 8 : 1);
    const int nv = ceil_div(vecs, lanes);
    const int smem = lanes == kThreads || partial == nullptr ? 0 : kThreads / lanes * 2 * width * 4;
    const T *xt = static_cast<const T*>(x), *gt = static_cast<const T*>(dy);
    T* o = static_cast<T*>(dx);
    launch_begin(kKindNormBwd, s);
    auto go = [&](auto kernel) {
        kernel<<<parts, kThreads, smem, s>>>(xt, x_row, weight, mean, rstd, gt, dy_row, rows, width, lanes, o, partial);
    };
    constexpr int M = V == 1 ? 4 : 1;
    if (nv <= 1 * M) go(norm_backward_kernel<T, V, 1 * M>);
    else if (nv <= 2 * M) go(norm_backward_kernel<T, V, 2 * M>);
    else if (nv <= 4 * M) go(norm_backward_kernel<T, V, 4 * M>);
    else
        norm_backward_wide_kernel<T><<<parts, kThreads, 0, s>>>(xt, x_row, weight, mean, rstd, gt, dy_row, rows, width, o,
                                                                partial);
    return launch_end(kKindNormBwd, s);
}

template <typename T>
int forward_type(const void* x, int64_t x_row, const float* weight, const float* bias, float eps, int64_t rows, int width,
                 void* y, float* mean, float* rstd, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (width % V == 0 && x_row % V == 0 && on(x, 16) && on(y, 16))
        return forward_of<T, V>(x, x_row, weight, bias, eps, rows, width, y, mean, rstd, s);
    return forward_of<T, 1>(x, x_row, weight, bias, eps, rows, width, y, mean, rstd, s);
}

template <typename T>
int backward_type(const void* x, int64_t x_row, const float* weight, const float* mean, const float* rstd, const void* dy,
                  int64_t dy_row, int64_t rows, int width, void* dx, float* partial, int parts, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (width % V == 0 && x_row % V == 0 && dy_row % V == 0 && on(x, 16) && on(dy, 16) && on(dx, 16))
        return backward_of<T, V>(x, x_row, weight, mean, rstd, dy, dy_row, rows, width, dx, partial, parts, s);
    return backward_of<T, 1>(x, x_row, weight, mean, rstd, dy, dy_row, rows, width, dx, partial, parts, s);
}

}  // namespace

int launch_layer_norm_forward(int dtype, const void* x, int64_t x_row, const float* weight, const float* bias, float eps,
                              int64_t rows, int width, void* y, float* mean, float* rstd, cudaStream_t s) {
    if (dtype == SSD_BF16) return forward_type<__nv_bfloat16>(x, x_row, weight, bias, eps, rows, width, y, mean, rstd, s);
    if (dtype == SSD_F16) return forward_type<__half>(x, x_row, weight, bias, eps, rows, width, y, mean, rstd, s);
    return forward_type<float>(x, x_row, weight, bias, eps, rows, width, y, mean, rstd, s);
}

// Blocks of the backward kernel: two per SM, or one per eight rows where there are few.
int layer_norm_parts(int64_t rows, int width, int sms) {
    (void)width;
    const int64_t want = ceil_div64(rows, 8);
    return (int)(want < 2 * sms ? want : 2 * sms);
}

int launch_layer_norm_backward(int dtype, const void* x, int64_t x_row, const float* weight, const float* mean,
                               const float* rstd, const void* dy, int64_t dy_row, int64_t rows, int width, void* dx,
                               float* dweight, float* dbias, float* partial, int parts, cudaStream_t s) {
    int r;
    if (dtype == SSD_BF16)
        r = backward_type<__nv_bfloat16>(x, x_row, weight, mean, rstd, dy, dy_row, rows, width, dx, partial, parts, s);
    else if (dtype == SSD_F16)
        r = backward_type<__half>(x, x_row, weight, mean, rstd, dy, dy_row, rows, width, dx, partial, parts, s);
    else
        r = backward_type<float>(x, x_row, weight, mean, rstd, dy, dy_row, rows, width, dx, partial, parts, s);
    if (r != SSD_OK || partial == nullptr) return r;
    launch_begin(kKindNormBwd, s);
    norm_reduce_kernel<<<ceil_div(2 * width, 32), 256, 0, s>>>(partial, parts, width, dweight, dbias);
    return launch_end(kKindNormBwd, s);
}

}  // namespace ssd
