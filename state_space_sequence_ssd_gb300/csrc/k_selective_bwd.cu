// k_selective_bwd.cu -- the gradients of the selective scan (k_selective.cu has the forward recurrence).  With
// a[t][n] = exp(dt[t] A[n]), g = dLoss/dy before the gate, and lam[t] the gradient of the state after token t:
//
//   lam[t][n] = C[t][n] g[t] + a[t+1][n] lam[t+1][n]          (+ dfinal after the last token)
//   dx[t]  = dt sum_n lam B + D g          ddt[t] = sum_n A a h[t-1] lam + x sum_n lam B   (times the softplus' slope)
//   dB[t][n] = sum_c lam dt x              dC[t][n] = sum_c g h[t]           (over the channels of a group)
//   dA[n] = sum_t dt a h[t-1] lam          dD = sum_t g x          dz[t] = dy y0 d(z sigmoid z)/dz,  y0 ungated
//
// The sequence is cut into blocks of kBlock tokens.  One kernel forms every block's own end state and its own
// gradient at its start, from zero; a hop carries both across the blocks (forward and backward in time); the main
// kernel then works on every block by itself, from its true start state and end gradient.  Inside a block the
// states are recomputed in runs of kRun tokens from a checkpoint at each run's start, since only the decay, not its
// inverse, is stable.  No atomics: sums over channels and blocks are written as rows of partial sums and added in a
// fixed order.
#include "selective.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kBlock = 64;  // tokens of a block
constexpr int kRun = 8;     // tokens whose states are held in registers
constexpr float kLn2 = 0.6931471805599453f;

template <int LP>
struct Blk {
    static constexpr int CW = 32 / LP, CC = kWarps * CW, N4 = 4 * LP, CV = CC / 4;
    static constexpr int XI = (kBlock * CV + kThreads - 1) / kThreads;
    // shared memory, in floats
    static constexpr int OFF_B = 4 * kBlock * CC;                 // (dt, dt x, g, -) per token and channel, then B
    static constexpr int OFF_C = OFF_B + kBlock * N4;
    static constexpr int OFF_SB = OFF_C + kBlock * N4;            // sum_n lam B, sum_n A a h lam, y per token and channel
    static constexpr int OFF_CK = OFF_SB + 3 * kBlock * CC;       // checkpoints, four floats per thread and run
    static constexpr int OFF_RED = OFF_CK + 4 * kThreads * (kBlock / kRun);
    static constexpr int FLOATS = OFF_RED + kWarps * kRun * 2 * N4;
};

template <typename T>
struct Row {  // where a block's tokens and channels are
    const T *x, *dt, *z, *B, *C, *dy;
    int b, grp, c0, nc, tb, te, len;  // c0: first channel; nc: channels of this block; tokens tb .. te - 1
};

template <typename T, int LP>
__device__ __forceinline__ Row<T> row_of(const SelectiveArgs& a, const void* dy) {
    using K = Blk<LP>;
    Row<T> r;
    const int per = a.channels / a.ngroups, tiles = (per + K::CC - 1) / K::CC;
    r.grp = blockIdx.x / tiles;
    const int cb = (blockIdx.x % tiles) * K::CC;
    r.c0 = r.grp * per + cb;
    r.nc = min(K::CC, per - cb);
    r.b = blockIdx.z;
    r.tb = blockIdx.y * kBlock;
    r.te = min(r.tb + kBlock, a.seqlen);
    r.len = row_length(a.lengths, r.b, a.seqlen);
    r.x = static_cast<const T*>(a.x) + r.b * a.x_batch + r.c0;
    r.dt = static_cast<const T*>(a.dt) + r.b * a.dt_batch + r.c0;
    r.z = a.z == nullptr ? nullptr : static_cast<const T*>(a.z) + r.b * a.z_batch + r.c0;
    r.B = static_cast<const T*>(a.B) + r.b * a.B_batch + (int64_t)r.grp * a.dstate;
    r.C = static_cast<const T*>(a.C) + r.b * a.C_batch + (int64_t)r.grp * a.dstate;
    r.dy = static_cast<const T*>(dy) + (int64_t)r.b * a.seqlen * a.channels + r.c0;
    return r;
}

// The block's tokens into shared memory: (dt, dt x, g, -) per token and channel, B and C as float32; zero past the
// length.  Returns this thread's sums of dt over its tokens, per channel of its vector.
template <typename T, int LP>
__device__ __forceinline__ void stage_block(const SelectiveArgs& a, const Row<T>& r, float* sm, bool vec, bool vecb,
                                            float (&dsum)[4]) {
    using K = Blk<LP>;
    const int tid = threadIdx.x, v0 = tid % K::CV;
    float4* s_q = reinterpret_cast<float4*>(sm);
    float bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        bias[e] = (a.dto.bias != nullptr && 4 * v0 + e < r.nc) ? a.dto.bias[r.c0 + 4 * v0 + e] : 0.f;
        dsum[e] = 0.f;
    }
#pragma unroll 2
    for (int i = 0; i < K::XI; ++i) {
        const int idx = tid + i * kThreads, t = r.tb + idx / K::CV;
        if (idx >= kBlock * K::CV) break;
        const bool live = t < r.len && t < r.te;
        const int valid = live ? max(0, r.nc - 4 * v0) : 0;
        const Vec<T, 4> x = load_vec<T, 4>(r.x + t * a.x_token + 4 * v0, valid, vec);
        const Vec<T, 4> d = load_vec<T, 4>(r.dt + t * a.dt_token + 4 * v0, valid, vec);
        const Vec<T, 4> dy = load_vec<T, 4>(r.dy + (int64_t)t * a.channels + 4 * v0, valid, vec);
        Vec<T, 4> z;
        if (r.z != nullptr) z = load_vec<T, 4>(r.z + t * a.z_token + 4 * v0, valid, vec);
        float dt[4], g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dt[e] = d.get(e) + bias[e];
            g[e] = dy.get(e);
        }
        effective(dt, a.dto);
        if (r.z != nullptr) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float zv = z.get(e);
                g[e] *= zv * sigmoid(zv);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dt[e] = live ? dt[e] : 0.f;
            s_q[(idx / K::CV) * K::CC + 4 * v0 + e] = make_float4(dt[e], dt[e] * x.get(e), g[e], 0.f);
            dsum[e] += dt[e];
        }
    }
    float4 *s_B = reinterpret_cast<float4*>(sm + K::OFF_B), *s_C = reinterpret_cast<float4*>(sm + K::OFF_C);
    for (int idx = tid; idx < kBlock * LP; idx += kThreads) {
        const int t = r.tb + idx / LP, n = 4 * (idx % LP);
        const int valid = (t < r.len && t < r.te) ? max(0, a.dstate - n) : 0;
        const Vec<T, 4> B = load_vec<T, 4>(r.B + t * a.B_token + n, valid, vecb);
        const Vec<T, 4> C = load_vec<T, 4>(r.C + t * a.C_token + n, valid, vecb);
        s_B[idx] = make_float4(B.get(0), B.get(1), B.get(2), B.get(3));
        s_C[idx] = make_float4(C.get(0), C.get(1), C.get(2), C.get(3));
    }
}

__device__ __forceinline__ void read4(const float* p, int valid, f32x2& lo, f32x2& hi, float scale = 1.f) {
    const Vec<float, 4> v = load_vec<float, 4, true>(p, valid, false);
    lo = pk(v.get(0) * scale, v.get(1) * scale);
    hi = pk(v.get(2) * scale, v.get(3) * scale);
}
__device__ __forceinline__ void write4(float* p, int valid, f32x2 lo, f32x2 hi) {
    float v[4];
    unpk(lo, v[0], v[1]);
    unpk(hi, v[2], v[3]);
    store_vec<float, 4>(p, Vec<float, 4>::of(v), valid, false);
}

// Every block's own end state (from zero) into hops[k + 1], its own gradient at its start into mus[k - 1] (block 0's
// into `nu0`), and its sum of dt.
template <typename T, int LP>
__global__ void __launch_bounds__(kThreads) selective_terms_kernel(SelectiveArgs a, const T* __restrict__ dy, int nblocks,
                                                                   float* __restrict__ hops, float* __restrict__ mus,
                                                                   float* __restrict__ nu0, float* __restrict__ dtsum,
                                                                   bool vec, bool vecb) {
    using K = Blk<LP>;
    extern __shared__ __align__(16) float sm[];
    const Row<T> r = row_of<T, LP>(a, dy);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.dstate, k = blockIdx.y;
    const int cl = warp * K::CW + lane / LP, q = lane % LP;
    const bool mine = cl < r.nc;
    const int nvalid = mine ? max(0, min(4, N - 4 * q)) : 0;
    const int64_t at = (mine ? (int64_t)(r.c0 + cl) : 0) * N + 4 * q, n = (int64_t)a.channels * N;
    float dsum[4];
    stage_block<T, LP>(a, r, sm, vec, vecb, dsum);
    f32x2 A01, A23, h01 = 0ull, h23 = 0ull, v01 = 0ull, v23 = 0ull, p01 = pk(1.f, 1.f), p23 = p01;
    read4(a.A + at, nvalid, A01, A23, kLog2e);
    __syncthreads();
    const float4 *s_q = reinterpret_cast<const float4*>(sm) + cl, *s_B = reinterpret_cast<const float4*>(sm + K::OFF_B) + q,
                 *s_C = reinterpret_cast<const float4*>(sm + K::OFF_C) + q;
    const int steps = min(r.te, r.len) - r.tb;
#pragma unroll 4
    for (int t = 0; t < steps; ++t) {
        const float4 d = s_q[t * K::CC], B = s_B[t * LP], C = s_C[t * LP];
        const f32x2 dd = pk(d.x, d.x), dx = pk(d.y, d.y), g = pk(d.z, d.z);
        const f32x2 a01 = exp2_2(mul2(dd, A01)), a23 = exp2_2(mul2(dd, A23));
        h01 = fma2(a01, h01, mul2(dx, pk(B.x, B.y)));
        h23 = fma2(a23, h23, mul2(dx, pk(B.z, B.w)));
        p01 = mul2(p01, a01);
        p23 = mul2(p23, a23);
        v01 = fma2(p01, mul2(g, pk(C.x, C.y)), v01);
        v23 = fma2(p23, mul2(g, pk(C.z, C.w)), v23);
    }
    const int64_t row = ((int64_t)r.b * nblocks + k) * n;
    if (k + 1 < nblocks) write4(hops + row + n + at, nvalid, h01, h23);
    if (k > 0) write4(mus + row - n + at, nvalid, v01, v23);
    else write4(nu0 + r.b * n + at, nvalid, v01, v23);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) sm[(tid / K::CV) * K::CC + 4 * (tid % K::CV) + e] = dsum[e];
    __syncthreads();
    for (int c = tid; c < r.nc; c += kThreads) {
        float s = 0.f;
        for (int i = 0; i < kThreads / K::CV; ++i) s += sm[i * K::CC + c];
        dtsum[((int64_t)r.b * nblocks + k) * a.channels + r.c0 + c] = s;
    }
}

// hops[k]: the state that block k starts from; mus[k]: the gradient that reaches the state after block k from later
// tokens; dinit.
__global__ void __launch_bounds__(256) selective_hops_kernel(const float* __restrict__ A, const float* __restrict__ init,
                                                             const float* __restrict__ dfinal, int channels, int dstate,
                                                             int nblocks, float* __restrict__ hops, float* __restrict__ mus,
                                                             const float* __restrict__ nu0, const float* __restrict__ dtsum,
                                                             float* __restrict__ dinit) {
    const int64_t n = (int64_t)channels * dstate, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int b = blockIdx.y;
    if (i >= n) return;
    const float A2 = A[i] * kLog2e;
    const float* dp = dtsum + (int64_t)b * nblocks * channels + i / dstate;
    if (blockIdx.z == 0) {
        float* hp = hops + b * n * nblocks + i;
        float h = init != nullptr ? init[b * n + i] : 0.f;
        hp[0] = h;
#pragma unroll 4
        for (int k = 0; k + 1 < nblocks; ++k) {
            h = fmaf(exp2_fast(A2 * dp[(int64_t)k * channels]), h, hp[(k + 1) * n]);
            hp[(k + 1) * n] = h;
        }
    } else {
        float* mp = mus + b * n * nblocks + i;
        float m = dfinal != nullptr ? dfinal[b * n + i] : 0.f;
        mp[(nblocks - 1) * n] = m;
#pragma unroll 4
        for (int k = nblocks - 1; k > 0; --k) {
            m = fmaf(exp2_fast(A2 * dp[(int64_t)k * channels]), m, mp[(k - 1) * n]);
            mp[(k - 1) * n] = m;
        }
        if (dinit != nullptr) dinit[b * n + i] = fmaf(exp2_fast(A2 * dp[0]), m, nu0[b * n + i]);
    }
}

template <typename T, int LP>
__global__ void __launch_bounds__(kThreads) selective_block_kernel(SelectiveArgs a, const T* __restrict__ dy, int nblocks,
                                                                   float* __restrict__ hops, const float* __restrict__ mus,
                                                                   T* __restrict__ dx, T* __restrict__ ddt,
                                                                   T* __restrict__ dz, float* __restrict__ dbc,
                                                                   float* __restrict__ chan, bool vec, bool vecb) {
    using K = Blk<LP>;
    extern __shared__ __align__(16) float sm[];
    const Row<T> r = row_of<T, LP>(a, dy);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.dstate, k = blockIdx.y;
    const int cl = warp * K::CW + lane / LP, q = lane % LP;
    const bool mine = cl < r.nc;
    const int nvalid = mine ? max(0, min(4, N - 4 * q)) : 0;
    const int64_t at = (mine ? (int64_t)(r.c0 + cl) : 0) * N + 4 * q, n = (int64_t)a.channels * N;
    const int64_t row = ((int64_t)r.b * nblocks + k) * n;
    float unused[4];
    stage_block<T, LP>(a, r, sm, vec, vecb, unused);
    f32x2 A01, A23, h01, h23, m01, m23, dA01 = 0ull, dA23 = 0ull;
    read4(a.A + at, nvalid, A01, A23, kLog2e);
    read4(hops + row + at, nvalid, h01, h23);
    read4(mus + row + at, nvalid, m01, m23);
    __syncthreads();
    const float4 *s_q = reinterpret_cast<const float4*>(sm) + cl, *s_B = reinterpret_cast<const float4*>(sm + K::OFF_B) + q,
                 *s_C = reinterpret_cast<const float4*>(sm + K::OFF_C) + q;
    float *s_sb = sm + K::OFF_SB, *s_sa = s_sb + kBlock * K::CC, *s_y = s_sa + kBlock * K::CC;
    ulonglong2* ck = reinterpret_cast<ulonglong2*>(sm + K::OFF_CK) + tid;
    float* s_red = sm + K::OFF_RED;
    const int steps = max(0, min(r.te, r.len) - r.tb);
    const int runs = (steps + kRun - 1) / kRun;  // the tokens past the length are zeros: they change nothing
    // forward: a checkpoint per run
    for (int j = 0; j < runs; ++j) {
        ck[j * kThreads] = make_ulonglong2(h01, h23);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const float4 d = s_q[(j * kRun + i) * K::CC], B = s_B[(j * kRun + i) * LP];
            const f32x2 dd = pk(d.x, d.x), dtx = pk(d.y, d.y);
            h01 = fma2(exp2_2(mul2(dd, A01)), h01, mul2(dtx, pk(B.x, B.y)));
            h23 = fma2(exp2_2(mul2(dd, A23)), h23, mul2(dtx, pk(B.z, B.w)));
        }
    }
    // backward, run by run
    for (int j = runs - 1; j >= 0; --j) {
        f32x2 H01[kRun + 1], H23[kRun + 1], a01[kRun], a23[kRun];
        const ulonglong2 c0 = ck[j * kThreads];
        H01[0] = c0.x;
        H23[0] = c0.y;
        float ys[kRun], sb[kRun], sa[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int t = j * kRun + i;
            const float4 d = s_q[t * K::CC], B = s_B[t * LP], C = s_C[t * LP];
            const f32x2 dd = pk(d.x, d.x), dtx = pk(d.y, d.y);
            a01[i] = exp2_2(mul2(dd, A01));
            a23[i] = exp2_2(mul2(dd, A23));
            H01[i + 1] = fma2(a01[i], H01[i], mul2(dtx, pk(B.x, B.y)));
            H23[i + 1] = fma2(a23[i], H23[i], mul2(dtx, pk(B.z, B.w)));
            ys[i] = sum2(fma2(pk(C.z, C.w), H23[i + 1], mul2(pk(C.x, C.y), H01[i + 1])));
        }
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
            const int t = j * kRun + i;
            const float4 d = s_q[t * K::CC], B = s_B[t * LP], C = s_C[t * LP];
            const f32x2 dd = pk(d.x, d.x), dtx = pk(d.y, d.y), g = pk(d.z, d.z);
            m01 = fma2(g, pk(C.x, C.y), m01);  // lam
            m23 = fma2(g, pk(C.z, C.w), m23);
            sb[i] = sum2(fma2(m23, pk(B.z, B.w), mul2(m01, pk(B.x, B.y))));
            float v[8];
            unpk(mul2(m01, dtx), v[0], v[1]);
            unpk(mul2(m23, dtx), v[2], v[3]);
            unpk(mul2(H01[i + 1], g), v[4], v[5]);
            unpk(mul2(H23[i + 1], g), v[6], v[7]);
            m01 = mul2(m01, a01[i]);
            m23 = mul2(m23, a23[i]);
            const f32x2 held01 = mul2(m01, H01[i]), held23 = mul2(m23, H23[i]);
            dA01 = fma2(held01, dd, dA01);
            dA23 = fma2(held23, dd, dA23);
            sa[i] = sum2(fma2(held23, A23, mul2(held01, A01)));
            // over the warp's channels: dB's four entries, then dC's
            int which = 0;
            fold_between<8, 16, LP>(v, lane, which);
            constexpr int LEFT = K::CW >= 8 ? 1 : 8 / K::CW;
            if ((lane / LP) % (K::CW >= 8 ? K::CW / 8 : 1) == 0) {
#pragma unroll
                for (int e = 0; e < LEFT; ++e) {
                    const int w = which + e;
                    s_red[((warp * kRun + i) * 2 + w / 4) * K::N4 + 4 * q + w % 4] = v[e];
                }
            }
        }
        // over the channel's lanes
        {
            int w = 0;
            fold_between<kRun, LP / 2, 1>(ys, lane, w);
            int w2 = 0;
            fold_between<kRun, LP / 2, 1>(sb, lane, w2);
            w2 = 0;
            fold_between<kRun, LP / 2, 1>(sa, lane, w2);
            constexpr int LEFT = LP >= kRun ? 1 : kRun / LP;
            if (q % (LP >= kRun ? LP / kRun : 1) == 0) {
#pragma unroll
                for (int e = 0; e < LEFT; ++e) {
                    const int at2 = (j * kRun + w + e) * K::CC + cl;
                    s_y[at2] = ys[e];
                    s_sb[at2] = sb[e];
                    s_sa[at2] = sa[e];
                }
            }
        }
        __syncthreads();
        for (int i = tid; i < kRun * 2 * N; i += kThreads) {
            const int tt = i / (2 * N), which = (i / N) % 2, e = i % N, t = r.tb + j * kRun + tt;
            if (t >= r.te) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += s_red[((w * kRun + tt) * 2 + which) * K::N4 + e];
            // dbc: (channel blocks of a group, batch, seqlen, ngroups, 2, dstate)
            const int per = a.channels / a.ngroups, tiles = (per + K::CC - 1) / K::CC;
            const int64_t tile = blockIdx.x % tiles;
            dbc[((((tile * a.batch + r.b) * a.seqlen + t) * a.ngroups + r.grp) * 2 + which) * N + e] = s;
        }
        __syncthreads();
    }
    // tokens past the last run have no gradient in B and C
    for (int i = tid; i < (r.te - r.tb - runs * kRun) * 2 * N; i += kThreads) {
        const int per = a.channels / a.ngroups, tiles = (per + K::CC - 1) / K::CC;
        const int64_t tile = blockIdx.x % tiles;
        const int t = r.tb + runs * kRun + i / (2 * N);
        dbc[(((tile * a.batch + r.b) * a.seqlen + t) * a.ngroups + r.grp) * 2 * N + i % (2 * N)] = 0.f;
    }
    write4(hops + row + at, nvalid, dA01, dA23);  // this block's part of dA, in place of its start state
    __syncthreads();
    // per token and channel
    const int v0 = tid % K::CV, valid = r.nc - 4 * v0;
    float dD[4] = {0.f, 0.f, 0.f, 0.f}, dbias[4] = {0.f, 0.f, 0.f, 0.f};
    if (valid > 0) {
        for (int i = 0; i < K::XI; ++i) {
            const int idx = tid + i * kThreads, t = r.tb + idx / K::CV;
            if (idx >= kBlock * K::CV || t >= r.te) break;
            const bool live = t < r.len;
            float ox[4], od[4], oz[4];
            const int got = live ? valid : 0;
            const Vec<T, 4> x = load_vec<T, 4>(r.x + t * a.x_token + 4 * v0, got, vec);
            const Vec<T, 4> d = load_vec<T, 4>(r.dt + t * a.dt_token + 4 * v0, got, vec);
            const Vec<T, 4> gy = load_vec<T, 4>(r.dy + (int64_t)t * a.channels + 4 * v0, got, vec);
            Vec<T, 4> z;
            if (r.z != nullptr) z = load_vec<T, 4>(r.z + t * a.z_token + 4 * v0, got, vec);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float fx = 0.f, fd = 0.f, fz = 0.f;
                if (live && e < valid) {
                    const int c = r.c0 + 4 * v0 + e, s = (idx / K::CV) * K::CC + 4 * v0 + e;
                    const float4 w = reinterpret_cast<const float4*>(sm)[s];  // dt, dt x, g
                    const float xv = x.get(e), Dc = a.D != nullptr ? a.D[c] : 0.f;
                    fx = fmaf(w.x, s_sb[s], Dc * w.z);
                    fd = fmaf(xv, s_sb[s], kLn2 * s_sa[s]);
                    const float raw = d.get(e) + (a.dto.bias != nullptr ? a.dto.bias[c] : 0.f);
                    if (a.dto.limit) {
                        const float soft = a.dto.softplus ? softplus(raw) : raw;
                        if (!(soft >= a.dto.lo && soft <= a.dto.hi)) fd = 0.f;
                    }
                    if (a.dto.softplus) fd *= sigmoid(raw);
                    dD[e] = fmaf(w.z, xv, dD[e]);
                    dbias[e] += fd;
                    if (r.z != nullptr) {
                        const float zv = z.get(e), sg = sigmoid(zv);
                        fz = gy.get(e) * fmaf(Dc, xv, s_y[s]) * sg * fmaf(zv, 1.f - sg, 1.f);
                    }
                }
                ox[e] = fx;
                od[e] = fd;
                oz[e] = fz;
            }
            const int64_t o = ((int64_t)r.b * a.seqlen + t) * a.channels + r.c0 + 4 * v0;
            store_vec<T, 4>(dx + o, Vec<T, 4>::of(ox), valid, vec);
            store_vec<T, 4>(ddt + o, Vec<T, 4>::of(od), valid, vec);
            if (dz != nullptr) store_vec<T, 4>(dz + o, Vec<T, 4>::of(oz), valid, vec);
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sm[(tid / K::CV) * 2 * K::CC + 4 * v0 + e] = dD[e];
        sm[(tid / K::CV) * 2 * K::CC + K::CC + 4 * v0 + e] = dbias[e];
    }
    __syncthreads();
    for (int i = tid; i < 2 * K::CC; i += kThreads) {
        if (i % K::CC >= r.nc) continue;
        float s = 0.f;
        for (int j = 0; j < kThreads / K::CV; ++j) s += sm[j * 2 * K::CC + i];
        chan[(((int64_t)r.b * nblocks + k) * 2 + i / K::CC) * a.channels + r.c0 + i % K::CC] = s;
    }
}

// out[i] = sum over rows of in[row * stride + i], i < n, in a fixed order: eight strided sums, then those eight.
__global__ void __launch_bounds__(256) column_sums_kernel(const float* __restrict__ in, int64_t stride, int rows, int64_t n,
                                                          float* __restrict__ out) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (i < n) {
#pragma unroll 8
        for (int r = warp; r < rows; r += 8) s += in[r * stride + i];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || i >= n) return;
    s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += part[q][lane];
    out[i] = s;
}

// dB and dC from the channel blocks' parts, (tiles, tokens and groups, 2, dstate), added in order
__global__ void __launch_bounds__(256) join_bc_kernel(const float* __restrict__ dbc, int tiles, int64_t rows, int dstate,
                                                      float* __restrict__ dB, float* __restrict__ dC) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, n = rows * 2 * dstate;
    if (i >= n) return;
    float s = 0.f;
#pragma unroll 8
    for (int t = 0; t < tiles; ++t) s += dbc[t * n + i];
    const int64_t row = i / (2 * dstate);
    const int e = (int)(i % (2 * dstate));
    if (e < dstate) dB[row * dstate + e] = s;
    else dC[row * dstate + e - dstate] = s;
}

int column_sums(const float* in, int64_t stride, int rows, int64_t n, float* out, cudaStream_t s) {
    launch_begin(kKindSelectiveBwd, s);
    column_sums_kernel<<<(unsigned)ceil_div64(n, 32), 256, 0, s>>>(in, stride, rows, n, out);
    return launch_end(kKindSelectiveBwd, s);
}

struct Parts {
    int nblocks, tiles;
    size_t hops, nu0, dtsum, chan, dbc;  // floats of each part
    size_t total() const { return 2 * hops + nu0 + dtsum + chan + dbc; }
};

Parts parts_of(const SelectiveArgs& a) {
    Parts p;
    const int cc = kWarps * 32 / selective_lanes(a.dstate);
    p.nblocks = ceil_div(a.seqlen, kBlock);
    p.tiles = ceil_div(a.channels / a.ngroups, cc);
    const size_t n = (size_t)a.channels * a.dstate, rows = (size_t)a.batch * p.nblocks;
    p.hops = rows * n;
    p.nu0 = a.batch * n;
    p.dtsum = rows * a.channels;
    p.chan = 2 * rows * a.channels;
    p.dbc = (size_t)p.tiles * a.batch * a.seqlen * a.ngroups * 2 * a.dstate;
    return p;
}

template <typename T, int LP>
int backward_lanes(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s) {
    using K = Blk<LP>;
    const Parts p = parts_of(a);
    float *hops = ws, *mus = hops + p.hops, *nu0 = mus + p.hops, *dtsum = nu0 + p.nu0, *chan = dtsum + p.dtsum,
          *dbc = chan + p.chan;
    const T* dy = static_cast<const T*>(g.dy);
    const bool vec = rows_of_four(a, g.dx, g.ddt, sizeof(T)) && aligned_to(g.dy, 4 * sizeof(T)) &&
                     aligned_to(g.dz, 4 * sizeof(T)) && a.channels % 4 == 0;
    const bool vecb = states_of_four(a, sizeof(T));
    const int smem = K::FLOATS * 4;
    const dim3 grid(a.ngroups * p.tiles, p.nblocks, a.batch);
    const int64_t n = (int64_t)a.channels * a.dstate;
    int r = ensure_smem_limit(reinterpret_cast<const void*>(selective_terms_kernel<T, LP>), smem);
    if (r == SSD_OK) r = ensure_smem_limit(reinterpret_cast<const void*>(selective_block_kernel<T, LP>), smem);
    if (r != SSD_OK) return r;
    launch_begin(kKindSelectiveBwd, s);
    selective_terms_kernel<T, LP><<<grid, kThreads, smem, s>>>(a, dy, p.nblocks, hops, mus, nu0, dtsum, vec, vecb);
    r = launch_end(kKindSelectiveBwd, s);
    if (r != SSD_OK) return r;
    launch_begin(kKindSelectiveBwd, s);
    selective_hops_kernel<<<dim3((unsigned)ceil_div64(n, 256), a.batch, 2), 256, 0, s>>>(
        a.A, a.init, g.dfinal, a.channels, a.dstate, p.nblocks, hops, mus, nu0, dtsum, g.dinit);
    r = launch_end(kKindSelectiveBwd, s);
    if (r != SSD_OK) return r;
    launch_begin(kKindSelectiveBwd, s);
    selective_block_kernel<T, LP><<<grid, kThreads, smem, s>>>(a, dy, p.nblocks, hops, mus, static_cast<T*>(g.dx),
                                                               static_cast<T*>(g.ddt), static_cast<T*>(g.dz), dbc, chan, vec,
                                                               vecb);
    r = launch_end(kKindSelectiveBwd, s);
    const int rows = a.batch * p.nblocks;
    if (r == SSD_OK) r = column_sums(hops, n, rows, n, g.dA, s);
    if (r == SSD_OK && g.dD != nullptr) r = column_sums(chan, 2 * a.channels, rows, a.channels, g.dD, s);
    if (r == SSD_OK && g.ddt_bias != nullptr)
        r = column_sums(chan + a.channels, 2 * a.channels, rows, a.channels, g.ddt_bias, s);
    if (r != SSD_OK) return r;
    const int64_t tokens = (int64_t)a.batch * a.seqlen * a.ngroups;
    launch_begin(kKindSelectiveBwd, s);
    join_bc_kernel<<<(unsigned)ceil_div64(tokens * 2 * a.dstate, 256), 256, 0, s>>>(dbc, p.tiles, tokens, a.dstate, g.dB, g.dC);
    return launch_end(kKindSelectiveBwd, s);
}

template <typename T>
int backward_of(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s) {
    switch (selective_lanes(a.dstate)) {
        case 2: return backward_lanes<T, 2>(a, g, ws, s);
        case 4: return backward_lanes<T, 4>(a, g, ws, s);
        case 8: return backward_lanes<T, 8>(a, g, ws, s);
        case 16: return backward_lanes<T, 16>(a, g, ws, s);
        case 32: return backward_lanes<T, 32>(a, g, ws, s);
        default: return SSD_ERR_UNSUPPORTED;
    }
}

}  // namespace

size_t selective_backward_workspace(const SelectiveArgs& a) { return parts_of(a).total() * sizeof(float); }

int launch_selective_backward(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s) {
    if (a.dtype == SSD_BF16) return backward_of<__nv_bfloat16>(a, g, ws, s);
    if (a.dtype == SSD_F16) return backward_of<__half>(a, g, ws, s);
    return backward_of<float>(a, g, ws, s);
}

}  // namespace ssd
