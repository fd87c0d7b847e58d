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
#include "norm.cuh"

namespace ssd {
namespace {

// NV vectors of V columns per thread: thread `lane` holds columns (lane + lanes i) V ..  A block takes its rows and ends.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const T* __restrict__ x, int64_t x_row,
                                                                const float* __restrict__ weight,
                                                                const float* __restrict__ bias, float eps, int64_t rows,
                                                                int width, int lanes, T* __restrict__ y,
                                                                float* __restrict__ mean, float* __restrict__ rstd, bool vecw) {
    constexpr int P = (V + 1) / 2;
    __shared__ float2 buf[2][kThreads / 32];
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t row = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    const bool live = row < rows;
    const T* xr = x + (live ? row : 0) * x_row;
    const float inv = 1.f / (float)width;
    Vec<T, V> r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + lanes * i) * V;
        r[i] = load_vec<T, V>(xr + c, live ? width - c : 0, true);
    }
    f32x2 s2 = 0ull, q2 = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) s2 = add2(s2, r[i].pair(e));
    const float m = row_sum(sum2(s2), lanes, buf[0]) * inv;
    const f32x2 m2 = pk(-m, V > 1 ? -m : 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((lane + lanes * i) * V < width) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const f32x2 d = add2(r[i].pair(e), m2);
                q2 = fma2(d, d, q2);
            }
        }
    const float rs = rsqrtf(fmaf(row_sum(sum2(q2), lanes, buf[1]), inv, eps));
    if (!live) return;
    if (lane == 0) {
        if (mean != nullptr) mean[row] = m;
        if (rstd != nullptr) rstd[row] = rs;
    }
    T* yr = y + row * width;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + lanes * i) * V;
        if (c >= width) break;
        f32x2 o[P], w[P], b[P];
        load_columns<V>(weight, c, width, vecw, 1.f, w);
        load_columns<V>(bias, c, width, vecw, 0.f, b);
#pragma unroll
        for (int e = 0; e < P; ++e) o[e] = fma2(mul2(add2(r[i].pair(e), m2), pk(rs, rs)), w[e], b[e]);
        store_vec<T, V>(yr + c, Vec<T, V>::of_pairs(o), width - c, true);
    }
}

// The same for many rows, with vectors of 16 bytes: a resident grid whose blocks walk the rows, two neighbouring ones a
// thread, so that they share the reductions' barriers and the weight and bias that it holds.  A thread's pieces of the
// next rows are copied to shared memory that it alone reads, so that they need neither registers nor barriers while they
// are on their way.  At 8192 x 2048 of bfloat16 14.4 us where two sets of inputs take turns (part of them stays in L2), 16.7
// where they come from HBM (4.0 TB/s; a plain copy of as many bytes 12.3); the kernel above takes 19.3 where this takes
// 14.4, and at 30400 x 2048 63 where this takes 46 (5.4 TB/s).  Copies of one, three and four pairs of
// rows ahead took 3 to 7% longer than two, reading the weight again for each row 14%.
constexpr int kAhead = 2;  // pairs of rows
constexpr int resident(int nv) { return nv <= 2 ? 3 : 2; }  // blocks of an SM
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads, resident(NV)) norm_ring_kernel(const T* __restrict__ x, int64_t x_row,
                                                                const float* __restrict__ weight,
                                                                const float* __restrict__ bias, float eps, int64_t rows,
                                                                int width, int lanes, T* __restrict__ y,
                                                                float* __restrict__ mean, float* __restrict__ rstd, bool vecw) {
    constexpr int P = (V + 1) / 2, R = 2;
    constexpr bool HOLD = NV <= 2;  // weight and bias stay in registers
    __shared__ float2 buf[2][kThreads / 32];
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & (lanes - 1), per = kThreads / lanes;
    const float inv = 1.f / (float)width;
    uint4* ring = reinterpret_cast<uint4*>(smem) + threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * per * R;
    int64_t row = ((int64_t)blockIdx.x * per + threadIdx.x / lanes) * R;
    auto fetch = [&](int64_t r0, int turn) {
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + lanes * i) * V;
                const bool in = r0 + k < rows && c < width;
                copy16(ring + ((turn * R + k) * NV + i) * kThreads, in ? x + (r0 + k) * x_row + c : x, in);
            }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(row + k * step, k);
    f32x2 w[NV][P], b[NV][P];
    if (HOLD) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            load_columns<V>(weight, (lane + lanes * i) * V, width, vecw, 1.f, w[i]);
            load_columns<V>(bias, (lane + lanes * i) * V, width, vecw, 0.f, b[i]);
        }
    }
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * per * R; r0 < rows; r0 += step, row += step) {
        Vec<T, V> r[R][NV];
        copies_wait<kAhead - 1>();
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint4 u = ring[((turn * R + k) * NV + i) * kThreads];
                r[k][i].w[0] = u.x; r[k][i].w[1] = u.y; r[k][i].w[2] = u.z; r[k][i].w[3] = u.w;
            }
        float m[2], rs[2];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            f32x2 s = 0ull;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < P; ++e) s = add2(s, r[k][i].pair(e));
            m[k] = sum2(s) * inv;
        }
        fetch(row + kAhead * step, turn);
        if (++turn == kAhead) turn = 0;
        const float2 mm = row_sums(make_float2(m[0], m[1]), lanes, buf[0]);
        m[0] = mm.x;
        m[1] = mm.y;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const f32x2 m2 = pk(-m[k], -m[k]);
            f32x2 q = 0ull;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if ((lane + lanes * i) * V < width) {
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        const f32x2 d = add2(r[k][i].pair(e), m2);
                        q = fma2(d, d, q);
                    }
                }
            rs[k] = sum2(q) * inv;
        }
        const float2 qq = row_sums(make_float2(rs[0], rs[1]), lanes, buf[1]);
        rs[0] = rsqrtf(qq.x + eps);
        rs[1] = rsqrtf(qq.y + eps);
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (lane == 0 && row + k < rows) {
                if (mean != nullptr) mean[row + k] = m[k];
                if (rstd != nullptr) rstd[row + k] = rs[k];
            }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + lanes * i) * V;
            if (c >= width) break;
            if (!HOLD) {
                load_columns<V>(weight, c, width, vecw, 1.f, w[i]);
                load_columns<V>(bias, c, width, vecw, 0.f, b[i]);
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                f32x2 o[P];
#pragma unroll
                for (int e = 0; e < P; ++e)
                    o[e] = fma2(mul2(add2(r[k][i].pair(e), pk(-m[k], -m[k])), pk(rs[k], rs[k])), w[i][e], b[i][e]);
                store_vec<T, V>(y + (row + k) * width + c, Vec<T, V>::of_pairs(o), row + k < rows ? width - c : 0, true);
            }
        }
    }
    copies_wait<0>();
}

// Rows that do not fit the registers, a block each: read again (from L2) for each sum and the output.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_forward_wide_kernel(const T* __restrict__ x, int64_t x_row,
                                                                     const float* __restrict__ weight,
                                                                     const float* __restrict__ bias, float eps, int width,
                                                                     T* __restrict__ y, float* __restrict__ mean,
                                                                     float* __restrict__ rstd) {
    __shared__ float2 buf[2][kThreads / 32];
    const int64_t row = blockIdx.x;
    const T* xr = x + row * x_row;
    const float inv = 1.f / (float)width;
    float s = 0.f, q = 0.f;
#pragma unroll 8
    for (int c = threadIdx.x; c < width; c += kThreads) s += to_f32<T>(xr[c]);
    const float m = row_sum(s, kThreads, buf[0]) * inv;
#pragma unroll 8
    for (int c = threadIdx.x; c < width; c += kThreads) {
        const float d = to_f32<T>(xr[c]) - m;
        q = fmaf(d, d, q);
    }
    const float rs = rsqrtf(fmaf(row_sum(q, kThreads, buf[1]), inv, eps));
    if (threadIdx.x == 0) {
        if (mean != nullptr) mean[row] = m;
        if (rstd != nullptr) rstd[row] = rs;
    }
#pragma unroll 8
    for (int c = threadIdx.x; c < width; c += kThreads)
        y[row * width + c] = from_f32<T>(fmaf((to_f32<T>(xr[c]) - m) * rs, weight != nullptr ? weight[c] : 1.f,
                                              bias != nullptr ? bias[c] : 0.f));
}

// A block of `lanes` threads a row, kThreads / lanes rows at a time.  The thread's columns of dweight and dbias stay
// in registers while the block walks its rows, and the next rows' loads are in flight while a row is summed.  With the
// reduction 27.2 us at 8192 x 2048 of bfloat16 (a plain sum of two such tensors takes 15.7): bound by latency, with 52% of the
// issue slots used at 15 warps an SM, which the sums' registers allow.  Smaller parts of a row a thread (8 columns instead of 16) and more
// blocks took 39 us and more, loads three rows ahead through shared memory as long as these one row ahead.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const T* __restrict__ x, int64_t x_row,
                                                                 const float* __restrict__ weight,
                                                                 const float* __restrict__ mean,
                                                                 const float* __restrict__ rstd, const T* __restrict__ dy,
                                                                 int64_t dy_row, int64_t rows, int width, int lanes,
                                                                 T* __restrict__ dx, float* __restrict__ partial, bool vecw) {
    extern __shared__ float sums[];  // (kThreads / lanes) x 2 x width where rows share a block
    __shared__ float2 buf[2][kThreads / 32];
    const int lane = threadIdx.x & (lanes - 1), slot = threadIdx.x / lanes, per = kThreads / lanes;
    const float inv = 1.f / (float)width;
    constexpr int P = (V + 1) / 2;
    f32x2 w[NV][P], dw[NV][P], db[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_columns<V>(weight, (lane + lanes * i) * V, width, vecw, 1.f, w[i]);
#pragma unroll
        for (int e = 0; e < P; ++e) dw[i][e] = db[i][e] = 0ull;
    }
    Vec<T, V> nx[NV], ng[NV];
    float nm, nrs;
    auto fetch = [&](int64_t row) {
        const bool live = row < rows;
        const int64_t at = live ? row : 0;
        nm = live ? __ldg(mean + at) : 0.f;
        nrs = live ? __ldg(rstd + at) : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + lanes * i) * V;
            nx[i] = load_vec<T, V>(x + at * x_row + c, live ? width - c : 0, true);
            ng[i] = load_vec<T, V>(dy + at * dy_row + c, live ? width - c : 0, true);
        }
    };
    const int64_t step = (int64_t)gridDim.x * per;
    int64_t row = (int64_t)blockIdx.x * per + slot;
    fetch(row);
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < rows; r0 += step, row += step, turn ^= 1) {
        Vec<T, V> cx[NV], cg[NV];
        const float rs = nrs, minus = -nm;  // xhat = (x - mean) rstd: x rstd - (mean rstd) would shift the whole row by that product's rounding
        const f32x2 rs2 = pk(rs, rs);
        f32x2 s1 = 0ull, s2 = 0ull;
#pragma unroll
        for (int i = 0; i < NV; ++i) { cx[i] = nx[i]; cg[i] = ng[i]; }
        if (r0 + step < rows) fetch(row + step);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const f32x2 gy = cg[i].pair(e), xh = mul2(pair_plus(cx[i], e, minus), rs2);  // gy is zero past the row's end
                const f32x2 g = mul2(gy, w[i][e]);
                db[i][e] = add2(db[i][e], gy);
                dw[i][e] = fma2(gy, xh, dw[i][e]);
                s1 = add2(s1, g);
                s2 = fma2(g, xh, s2);
            }
        float2 s = make_float2(sum2(s1), sum2(s2));
        s = row_sums(s, lanes, buf[turn]);
        if (row >= rows) continue;
        const float k1 = -s.x * inv * rs, k2 = -s.y * inv * rs;
        T* o = dx + row * width;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + lanes * i) * V;
            if (c >= width) break;
            f32x2 out[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const f32x2 xh = mul2(pair_plus(cx[i], e, minus), rs2), g = mul2(cg[i].pair(e), w[i][e]);
                out[e] = fma2(g, rs2, fma2(xh, pk(k2, k2), pk(k1, k1)));
            }
            store_vec<T, V>(o + c, Vec<T, V>::of_pairs(out), width - c, true);
        }
    }
    if (partial == nullptr) return;
    float* out = partial + (int64_t)blockIdx.x * 2 * width;
    float* to = per == 1 ? out : sums + slot * 2 * width;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = (lane + lanes * i) * V + e;
            float a, b;
            unpk(dw[i][e / 2], a, b);
            if (c < width) to[c] = e & 1 ? b : a;
            unpk(db[i][e / 2], a, b);
            if (c < width) to[width + c] = e & 1 ? b : a;
        }
    if (per == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * width; c += kThreads) {
        float s = 0.f;
        for (int q = 0; q < per; ++q) s += sums[q * 2 * width + c];
        out[c] = s;
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
    __shared__ float2 buf[2][kThreads / 32];
    const float inv = 1.f / (float)width;
    int turn = 0;
    float* sum = partial == nullptr ? nullptr : partial + (int64_t)blockIdx.x * 2 * width;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T *xr = x + row * x_row, *gr = dy + row * dy_row;
        const float m = mean[row], rs = rstd[row];
        float2 s = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float gy = to_f32<T>(gr[c]), xh = (to_f32<T>(xr[c]) - m) * rs;
            const float g = gy * (weight != nullptr ? weight[c] : 1.f);
            if (sum != nullptr) {
                const bool first = row == blockIdx.x;
                sum[c] = first ? gy * xh : fmaf(gy, xh, sum[c]);
                sum[width + c] = first ? gy : sum[width + c] + gy;
            }
            s.x += g;
            s.y = fmaf(g, xh, s.y);
        }
        s = row_sums(s, kThreads, buf[turn]);
        turn ^= 1;
        const float s1 = s.x * inv, s2 = s.y * inv;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float g = to_f32<T>(gr[c]) * (weight != nullptr ? weight[c] : 1.f), xh = (to_f32<T>(xr[c]) - m) * rs;
            dx[row * width + c] = from_f32<T>(rs * (g - s1 - xh * s2));
        }
    }
}

// dweight and dbias from the blocks' rows of `partial`: kJoin strided sums, then those.  The rows lie in L2 and what counts
// is how many of them are on their way at once.  (`partial` is written while this kernel may already run, so it is neither
// const for the kernel nor read as such.)
constexpr int kJoin = 32;
__global__ void __launch_bounds__(32 * kJoin) norm_reduce_kernel(const float* partial, int parts, int width,
                                                          float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float part[kJoin][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;
    grid_dep_wait();
    float s = 0.f;
    const int columns = dbias != nullptr ? 2 * width : width;  // of a row that are wanted
    if (i < columns) {
#pragma unroll 8
        for (int r = warp; r < parts; r += kJoin) s += partial[(int64_t)r * 2 * width + i];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || i >= columns) return;
    s = 0.f;
#pragma unroll
    for (int q = 0; q < kJoin; ++q) s += part[q][lane];
    if (i < width) {
        if (dweight != nullptr) dweight[i] = s;
    } else {
        dbias[i - width] = s;
    }
}

template <typename T, int V>
int forward_of(const void* x, int64_t x_row, const float* weight, const float* bias, float eps, int64_t rows, int width,
               void* y, float* mean, float* rstd, cudaStream_t s) {
    constexpr int M = V == 1 ? 4 : 1;
    const int vecs = ceil_div(width, V);
    const int lanes = row_lanes(rows, vecs, 2 * M, 1);
    const int nv = ceil_div(vecs, lanes);
    const int64_t blocks = ceil_div64(rows, kThreads / lanes);
    const bool vecw = aligned_to(weight, 16) && aligned_to(bias, 16);
    const T* xt = static_cast<const T*>(x);
    T* yt = static_cast<T*>(y);
    if (blocks > 2147483647) return SSD_ERR_UNSUPPORTED;
    launch_begin(kKindNorm, s);
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)blocks, kThreads, 0, s>>>(xt, x_row, weight, bias, eps, rows, width, lanes, yt, mean, rstd, vecw);
    };
    if constexpr (sizeof(T) * V == 16) {
        // A resident grid pays from about 24 thousand values an SM: with one row a thread's group and with the walk 4.4 and
        // 4.8 us at 1216 x 2048 of bfloat16, 7.2 and 5.8 at 1824 x 2048, 5.1 and 6.2 at 304 x 8192, 9.0 and 7.0 at
        // 608 x 8192, 5.6 and 6.4 at 1216 x 2048 of float32, 9.1 and 8.8 at 2432 x 2048.
        if (rows * width >= kSms * 24576 && nv <= 4) {
            int r = SSD_OK;
            auto walk = [&](auto kernel, int held) {
                const int smem = kAhead * 2 * held * kThreads * 16;
                r = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
                const int64_t pairs = ceil_div64(rows, kThreads / lanes * 2), most = kSms * resident(held);
                if (r == SSD_OK)
                    kernel<<<(unsigned)(pairs < most ? pairs : most), kThreads, smem, s>>>(xt, x_row, weight, bias, eps, rows, width, lanes, yt, mean, rstd, vecw);
            };
            nv == 1 ? walk(norm_ring_kernel<T, V, 1>, 1) : nv == 2 ? walk(norm_ring_kernel<T, V, 2>, 2) : walk(norm_ring_kernel<T, V, 4>, 4);
            const int e = launch_end(kKindNorm, s);
            return r != SSD_OK ? r : e;
        }
    }
    if (nv <= 1 * M) go(norm_forward_kernel<T, V, 1 * M>);
    else if (nv <= 2 * M) go(norm_forward_kernel<T, V, 2 * M>);
    else if (nv <= 4 * M) go(norm_forward_kernel<T, V, 4 * M>);
    else if (nv <= 8 * M) go(norm_forward_kernel<T, V, 8 * M>);
    else
        norm_forward_wide_kernel<T><<<(unsigned)blocks, kThreads, 0, s>>>(xt, x_row, weight, bias, eps, width, yt, mean, rstd);
    return launch_end(kKindNorm, s);
}

template <typename T, int V>
int backward_of(const void* x, int64_t x_row, const float* weight, const float* mean, const float* rstd, const void* dy,
                int64_t dy_row, int64_t rows, int width, void* dx, float* partial, int parts, cudaStream_t s) {
    constexpr int M = V == 1 ? 4 : 1;
    const int vecs = ceil_div(width, V);
    const int lanes = row_lanes(rows, vecs, 2 * M, 32);
    const int nv = ceil_div(vecs, lanes);
    const int smem = lanes == kThreads || partial == nullptr ? 0 : kThreads / lanes * 2 * width * 4;
    const T *xt = static_cast<const T*>(x), *gt = static_cast<const T*>(dy);
    T* o = static_cast<T*>(dx);
    const bool vecw = aligned_to(weight, 16);
    launch_begin(kKindNormBwd, s);
    auto go = [&](auto kernel) {
        kernel<<<parts, kThreads, smem, s>>>(xt, x_row, weight, mean, rstd, gt, dy_row, rows, width, lanes, o, partial, vecw);
    };
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
    if (width % V == 0 && x_row % V == 0 && aligned_to(x, 16) && aligned_to(y, 16))
        return forward_of<T, V>(x, x_row, weight, bias, eps, rows, width, y, mean, rstd, s);
    return forward_of<T, 1>(x, x_row, weight, bias, eps, rows, width, y, mean, rstd, s);
}

template <typename T>
int backward_type(const void* x, int64_t x_row, const float* weight, const float* mean, const float* rstd, const void* dy,
                  int64_t dy_row, int64_t rows, int width, void* dx, float* partial, int parts, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (width % V == 0 && x_row % V == 0 && dy_row % V == 0 && aligned_to(x, 16) && aligned_to(dy, 16) && aligned_to(dx, 16))
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
int layer_norm_parts(int64_t rows, int sms) {
    const int64_t want = ceil_div64(rows, 8);
    return (int)(want < 2 * sms ? want : 2 * sms);
}

int launch_norm_sums(int kind, const float* partial, int parts, int width, float* dweight, float* dbias, cudaStream_t s) {
    launch_begin(kind, s);
    launch_dependent(norm_reduce_kernel, dim3(ceil_div(dbias != nullptr ? 2 * width : width, 32)), dim3(32 * kJoin), 0, s, partial, parts, width, dweight, dbias);
    return launch_end(kind, s);
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
    return launch_norm_sums(kKindNormBwd, partial, parts, width, dweight, dbias, s);
}

}  // namespace ssd
