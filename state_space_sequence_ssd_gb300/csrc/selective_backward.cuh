// selective_backward.cuh -- the gradients of the selective scan (selective_forward.cuh has the forward recurrence), compiled
// once per element type: k_selective_bwd_bf16.cu, k_selective_bwd_f16.cu, k_selective_bwd_f32.cu.  With
// a[t][n] = exp(dt[t] A[n]), g = dLoss/dy before the gate, and lam[t] the gradient of the state after token t:
//
//   lam[t][n] = C[t][n] g[t] + a[t+1][n] lam[t+1][n]          (+ dfinal after the last token)
//   dx[t]  = dt sum_n lam B + D g          ddt[t] = sum_n A a h[t-1] lam + x sum_n lam B   (times the softplus' slope)
//   dB[t][n] = sum_c lam dt x              dC[t][n] = sum_c g h[t]           (over the channels of a group)
//   dA[n] = sum_t dt a h[t-1] lam          dD = sum_t g x          dz[t] = dy y0 d(z sigmoid z)/dz,  y0 ungated
//
// The sequence is cut into blocks of 32 or 16 tokens.  One kernel forms every block's own end state and its own
// gradient at its start, from zero; a hop carries both across the blocks (forward and backward in time); the main
// kernel then works on every block by itself, from its true start state and end gradient.  Inside a block the
// states are recomputed in runs of kRun tokens from a checkpoint at each run's start, since only the decay, not its
// inverse, is stable.  No atomics: sums over channels and blocks are written as rows of partial sums and added in a
// fixed order, by one launch for all of them.  At 2 x 4096 x 2048 x 16 of bfloat16 500 us, about 130 of them for the
// blocks' own terms: 240 registers a thread leave the main kernel two warps on an SM quarter and 48% of the issue slots.
//
// A lane holds four state entries of four neighbouring channels and LP lanes share a channel: shared memory returns 128
// bytes a clock to the registers, broadcast or not, and with one channel a lane the operands of an entry (32 bytes over
// the passes) took 32 clocks where the arithmetic takes 20.  The sums over channels, dB and dC, are formed over a lane's
// four first, so that the exchange between lanes carries a quarter.  The packed pairs are two channels.
#pragma once

#include "selective.cuh"

namespace ssd {
namespace {

constexpr int kRun = 8;     // tokens between checkpoints
constexpr int kHeld = 4;    // tokens whose states and decays are in registers
constexpr float kLn2 = 0.6931471805599453f;

template <int LP, int BLOCK>  // BLOCK: tokens of a block
struct Blk {
    static constexpr int NP = 4 * LP;                // entries, padded
    static constexpr int CONV = LP;                  // tokens that the block's threads convert at once
    static constexpr int CONVS = BLOCK / CONV;
    static_assert(CONVS > 0, "tokens for every thread");
    static constexpr int channels(int threads) { return 4 * threads / LP; }
    // shared memory in floats: dt, dt x (later sum lam B), g (later sum A a h lam), y per token and channel; B, C; the
    // warps' parts of dB and dC of a run; checkpoints, sixteen floats per thread and run
    static constexpr int floats(int threads) {
        return 4 * BLOCK * channels(threads) + 2 * BLOCK * NP + threads / 32 * kRun * 2 * NP + 16 * threads * (BLOCK / kRun);
    }
    static constexpr int floats_terms(int threads) { return 3 * BLOCK * channels(threads) + 2 * BLOCK * NP; }
};

template <typename T>
struct Rows {  // where a block's tokens and channels are
    const T *x, *dt, *z, *B, *C, *dy;
    int b, grp, tile, tiles, c0, nc, tb, te, last;  // c0: first channel, of nc; tokens tb .. te - 1, live ones before last
};

template <typename T, int BLOCK>
__device__ __forceinline__ Rows<T> rows_at(const SelectiveArgs& a, const void* dy, int cc) {
    Rows<T> r;
    const int per = a.channels / a.ngroups;
    r.tiles = (per + cc - 1) / cc;
    r.grp = blockIdx.x / r.tiles;
    r.tile = blockIdx.x % r.tiles;
    r.c0 = r.grp * per + r.tile * cc;
    r.nc = min(cc, per - r.tile * cc);
    r.b = blockIdx.z;
    r.tb = blockIdx.y * BLOCK;
    r.te = min(r.tb + BLOCK, a.seqlen);
    r.last = min(r.te, row_length(a.lengths, r.b, a.seqlen));
    r.x = static_cast<const T*>(a.x) + r.b * a.x_batch + r.c0;
    r.dt = static_cast<const T*>(a.dt) + r.b * a.dt_batch + r.c0;
    r.z = a.z == nullptr ? nullptr : static_cast<const T*>(a.z) + r.b * a.z_batch + r.c0;
    r.B = static_cast<const T*>(a.B) + r.b * a.B_batch + (int64_t)r.grp * a.dstate;
    r.C = static_cast<const T*>(a.C) + r.b * a.C_batch + (int64_t)r.grp * a.dstate;
    r.dy = static_cast<const T*>(dy) + (int64_t)r.b * a.seqlen * a.channels + r.c0;
    return r;
}

// Four tokens' vectors of x, dt, dy and z of a thread (tokens t0 + i CONV, channels 4 v0 ..), zeros where they are not
// live, and their dt with its bias and dLoss/d(ungated y).
template <typename T, int M>
struct Loaded {
    Vec<T, 4> x[M], d[M], dy[M], z[M];
};
template <typename T, int M, int CONV>
__device__ __forceinline__ Loaded<T, M> load_rows(const SelectiveArgs& a, const Rows<T>& r, int t0, int v0, bool vec) {
    Loaded<T, M> l;
    const int vc = r.nc - 4 * v0;
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int t = t0 + i * CONV, valid = t < r.last ? vc : 0;
        l.x[i] = load_vec<T, 4>(r.x + t * a.x_token + 4 * v0, valid, vec);
        l.d[i] = load_vec<T, 4>(r.dt + t * a.dt_token + 4 * v0, valid, vec);
        l.dy[i] = load_vec<T, 4>(r.dy + (int64_t)t * a.channels + 4 * v0, valid, vec);
        l.z[i] = r.z != nullptr ? load_vec<T, 4>(r.z + t * a.z_token + 4 * v0, valid, vec) : Vec<T, 4>::zero();
    }
    return l;
}

// The block's tokens into shared memory: dt, dt x and g per token and channel, B and C as float32; zero past the length.
// Returns zero, or NaN where this thread's part of dt x, g, B or C is not all finite.
template <typename T, int LP, int BLOCK>
__device__ __forceinline__ float stage_block(const SelectiveArgs& a, const Rows<T>& r, float* s_d, float* s_x, float* s_g,
                                             float* s_B, float* s_C, bool vec, bool vecb, float (&dsum)[4]) {
    using K = Blk<LP, BLOCK>;
    constexpr int M = K::CONVS < 8 ? K::CONVS : 8;
    const int tid = threadIdx.x, threads = blockDim.x, cc = K::channels(threads);
    const int v0 = tid % (cc / 4), w0 = tid / (cc / 4);
    float bias[4], undefined = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) dsum[e] = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < K::CONVS; i0 += M) {
        const int t0 = w0 + i0 * K::CONV;
        const Loaded<T, M> l = load_rows<T, M, K::CONV>(a, r, r.tb + t0, v0, vec);
        if (i0 == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                bias[e] = (a.dto.bias != nullptr && 4 * v0 + e < r.nc) ? __ldg(a.dto.bias + r.c0 + 4 * v0 + e) : 0.f;
            constexpr int R = 4;  // vectors of B and of C in flight
            for (int j0 = tid; j0 < BLOCK * LP; j0 += R * threads) {
                Vec<T, 4> B[R], C[R];
#pragma unroll
                for (int u = 0; u < R; ++u) {
                    const int j = j0 + u * threads, t = r.tb + j / LP, e = 4 * (j % LP);
                    const int valid = j < BLOCK * LP && t < r.last ? a.dstate - e : 0;
                    B[u] = load_vec<T, 4>(r.B + t * a.B_token + e, valid, vecb);
                    C[u] = load_vec<T, 4>(r.C + t * a.C_token + e, valid, vecb);
                }
#pragma unroll
                for (int u = 0; u < R; ++u) {
                    const int j = j0 + u * threads;
                    if (j < BLOCK * LP) {
                        *reinterpret_cast<float4*>(s_B + 4 * j) = make_float4(B[u].get(0), B[u].get(1), B[u].get(2), B[u].get(3));
                        *reinterpret_cast<float4*>(s_C + 4 * j) = make_float4(C[u].get(0), C[u].get(1), C[u].get(2), C[u].get(3));
#pragma unroll
                        for (int e = 0; e < 4; ++e) undefined = fmaf(0.f, C[u].get(e), fmaf(0.f, B[u].get(e), undefined));
                    }
                }
            }
        }
        constexpr int S = M < 4 ? M : 4;  // vectors converted side by side
#pragma unroll
        for (int s = 0; s < M; s += S) {
            float dt[4 * S], g[4 * S];
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dt[4 * i + e] = l.d[s + i].get(e) + bias[e];
                    g[4 * i + e] = l.dy[s + i].get(e);
                }
            effective<true>(dt, a.dto);
            if (r.z != nullptr) {
#pragma unroll
                for (int i = 0; i < S; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float zv = l.z[s + i].get(e);
                        g[4 * i + e] *= zv * sigmoid(zv);
                    }
            }
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const int t = t0 + (s + i) * K::CONV, at = t * cc + 4 * v0;
                const bool live = r.tb + t < r.last;
                float dx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dt[4 * i + e] = live ? dt[4 * i + e] : 0.f;
                    dx[e] = dt[4 * i + e] * l.x[s + i].get(e);
                    dsum[e] += dt[4 * i + e];
                    undefined = fmaf(0.f, g[4 * i + e], fmaf(0.f, dx[e], undefined));
                }
                *reinterpret_cast<float4*>(s_d + at) = make_float4(dt[4 * i], dt[4 * i + 1], dt[4 * i + 2], dt[4 * i + 3]);
                *reinterpret_cast<float4*>(s_x + at) = make_float4(dx[0], dx[1], dx[2], dx[3]);
                *reinterpret_cast<float4*>(s_g + at) = make_float4(g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]);
            }
        }
    }
    return undefined;
}

// A lane's four entries of four channels, as pairs of channels, from and to (channels, dstate) float32.
using Entries = f32x2[4][2];
__device__ __forceinline__ void read_entries(const float* p, int64_t c, int channels, int N, int e, float scale, Entries& o) {
    const bool four = N % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    Vec<float, 4> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load_vec<float, 4, true>(p + (c + i) * N + e, i < channels ? N - e : 0, four);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i][0] = pk(v[0].get(i) * scale, v[1].get(i) * scale);
        o[i][1] = pk(v[2].get(i) * scale, v[3].get(i) * scale);
    }
}
__device__ __forceinline__ void write_entries(float* p, int64_t c, int channels, int N, int e, const Entries& v) {
    const bool four = N % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    float o[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unpk(v[i][0], o[0][i], o[1][i]);
        unpk(v[i][1], o[2][i], o[3][i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        store_vec<float, 4>(p + (c + i) * N + e, Vec<float, 4>::of(o[i]), i < channels ? N - e : 0, four);
}
__device__ __forceinline__ void pairs_of(const float* p, f32x2 (&o)[2]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    o[0] = pk(v.x, v.y);
    o[1] = pk(v.z, v.w);
}
__device__ __forceinline__ void twice_of(const float* p, f32x2 (&o)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    o[0] = pk(v.x, v.x);
    o[1] = pk(v.y, v.y);
    o[2] = pk(v.z, v.z);
    o[3] = pk(v.w, v.w);
}

// Every block's own end state (from zero) into hops[k + 1], its own gradient at its start into mus[k - 1] (block 0's
// into `nu0`), and its sum of dt.
template <typename T, int LP, int BLOCK>
__global__ void __launch_bounds__(128, 3) selective_terms_kernel(SelectiveArgs a, const T* __restrict__ dy, int nblocks,
                                                                 float* __restrict__ hops, float* __restrict__ mus,
                                                                 float* __restrict__ nu0, float* __restrict__ dtsum,
                                                                 bool vec, bool vecb) {
    using K = Blk<LP, BLOCK>;
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x, threads = blockDim.x, cc = K::channels(threads), N = a.dstate, k = blockIdx.y;
    const Rows<T> r = rows_at<T, BLOCK>(a, dy, cc);
    const int qd = tid / LP, q = tid % LP, mine = r.nc - 4 * qd;
    const int64_t c = r.c0 + 4 * qd, n = (int64_t)a.channels * N;
    float *s_d = sm, *s_x = s_d + BLOCK * cc, *s_g = s_x + BLOCK * cc, *s_B = s_g + BLOCK * cc, *s_C = s_B + BLOCK * K::NP;
    float dsum[4];
    const float undefined = stage_block<T, LP, BLOCK>(a, r, s_d, s_x, s_g, s_B, s_C, vec, vecb, dsum);
    Entries A, h, v, p;
    read_entries(a.A, c, mine, N, 4 * q, kLog2e, A);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            h[e][j] = v[e][j] = 0ull;
            p[e][j] = pk(1.f, 1.f);
        }
    const bool finite = __syncthreads_or(undefined != 0.f) == 0;
    const int steps = r.last - r.tb;
#pragma unroll 2
    for (int t = 0; t < steps; ++t) {
        f32x2 d[2], x[2], g[2], B[4], C[4];
        pairs_of(s_d + t * cc + 4 * qd, d);
        pairs_of(s_x + t * cc + 4 * qd, x);
        pairs_of(s_g + t * cc + 4 * qd, g);
        twice_of(s_B + t * K::NP + 4 * q, B);
        twice_of(s_C + t * K::NP + 4 * q, C);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x2 w = exp2_2(mul2(d[j], A[e][j]));
                h[e][j] = fma2(w, h[e][j], mul2(x[j], B[e]));
                p[e][j] = mul2(p[e][j], w);
                v[e][j] = fma2(p[e][j], mul2(g[j], C[e]), v[e][j]);
            }
    }
    if (!finite) {
        // the products of decays may have rounded to zero, which an infinite g would make NaN: the gradient token by token
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e][0] = v[e][1] = 0ull;
#pragma unroll 1
        for (int t = steps - 1; t >= 0; --t) {
            f32x2 d[2], g[2], C[4];
            pairs_of(s_d + t * cc + 4 * qd, d);
            pairs_of(s_g + t * cc + 4 * qd, g);
            twice_of(s_C + t * K::NP + 4 * q, C);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < 2; ++j) v[e][j] = mul2(exp2_2(mul2(d[j], A[e][j])), fma2(g[j], C[e], v[e][j]));
        }
    }
    const int64_t row = ((int64_t)r.b * nblocks + k) * n;
    if (k + 1 < nblocks) write_entries(hops + row + n, c, mine, N, 4 * q, h);
    write_entries(k > 0 ? mus + row - n : nu0 + r.b * n, c, mine, N, 4 * q, v);
    __syncthreads();
    const int v0 = tid % (cc / 4), w0 = tid / (cc / 4);
    *reinterpret_cast<float4*>(sm + w0 * cc + 4 * v0) = make_float4(dsum[0], dsum[1], dsum[2], dsum[3]);
    __syncthreads();
    for (int i = tid; i < r.nc; i += threads) {
        float s = 0.f;
        for (int w = 0; w < K::CONV; ++w) s += sm[w * cc + i];
        dtsum[((int64_t)r.b * nblocks + k) * a.channels + r.c0 + i] = s;
    }
}

// A channel's sums over its lanes, to the token's row: each lane ends with one (or several) of its four channels.
template <int LP>
__device__ __forceinline__ void join_lanes(f32x2 lo, f32x2 hi, int lane, float* to) {
    float v[4];
    unpk(lo, v[0], v[1]);
    unpk(hi, v[2], v[3]);
    int which = 0;
    fold_between<4, LP / 2, 1>(v, lane, which);
    if (LP <= 4 || (lane & (LP / 4 > 0 ? LP / 4 - 1 : 0)) == 0) {
#pragma unroll
        for (int e = 0; e < (LP >= 4 ? 1 : 4 / LP); ++e) to[which + e] = v[e];
    }
}
// Four values over the warp's channels, to a lane's entries of a token's row of dB or dC.
template <int LP>
__device__ __forceinline__ void join_warp(float (&v)[4], int lane, float* to) {
    constexpr int CW = 32 / LP, LEFT = CW >= 4 ? 1 : 4 / CW;
    int which = 0;
    fold_between<4, 16, LP>(v, lane, which);
    if (CW <= 4 || ((lane / LP) & (CW / 4 > 0 ? CW / 4 - 1 : 0)) == 0) {
#pragma unroll
        for (int e = 0; e < LEFT; ++e) to[which + e] = v[e];
    }
}
// A token's dt, dt x, g, B and C for a lane's channels and entries; loaded a token ahead, so that no load waits behind a
// store it might meet.
struct Operands {
    float4 d, x, g, B, C;
};
template <int LP>
struct Lane {
    float *s_d, *s_x, *s_g, *s_B, *s_C;
    int cc, qd, q;
    static constexpr int NP = 4 * LP;
    __device__ __forceinline__ Operands operands(int t) const {
        auto at = [](const float* p) { return *reinterpret_cast<const float4*>(p); };
        return Operands{at(s_d + t * cc + 4 * qd), at(s_x + t * cc + 4 * qd), at(s_g + t * cc + 4 * qd), at(s_B + t * NP + 4 * q),
                        at(s_C + t * NP + 4 * q)};
    }
    __device__ __forceinline__ void advance(int t, const Entries& A, Entries& h) const {  // the states over token t
        f32x2 d[2], x[2], B[4];
        pairs_of(s_d + t * cc + 4 * qd, d);
        pairs_of(s_x + t * cc + 4 * qd, x);
        twice_of(s_B + t * NP + 4 * q, B);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < 2; ++j) h[e][j] = fma2(exp2_2(mul2(d[j], A[e][j])), h[e][j], mul2(x[j], B[e]));
    }
};

// The tokens of one run, last to first, each by itself from the run's checkpoint; y, red: this lane's places in the rows of
// y and of the warp's parts of dB and dC.  Entries past dstate, channels past the group's last and tokens past the length are
// zeros that add nothing -- unless they meet an infinity, zero times which is NaN: one of the token's other factors, or one in a
// state that an earlier token left.  So the runs of a block that holds an infinity or a NaN come here, where such zeros are left
// out of the sums; the same roundings otherwise.  Few registers count here, not time: kernels that have this beside their
// other runs take 5% longer (520 us against 497 at 2 x 4096 x 2000 x 16), so only shapes with padding do.
template <int LP>
__device__ __forceinline__ void alone(const Lane<LP> at, const ulonglong2* ck, int first, int end, int entries, int channels,
                                   float* y_row, float* red, const Entries& A, Entries& m, Entries& dA) {
    const int lane = threadIdx.x & 31, threads = blockDim.x;
    auto entry = [&](int e, f32x2 u, f32x2 v, f32x2 s) { return e < entries ? fma2(u, v, s) : s; };
    auto over_channels = [&](const f32x2 (&u)[2], const f32x2 (&v)[2]) {
        float s[2], p[2];
        unpk(mul2(u[0], v[0]), s[0], s[1]);
        s[0] = channels > 0 ? s[0] : 0.f;
        s[1] = channels > 1 ? s[1] : 0.f;
        unpk(fma2(u[1], v[1], pk(s[0], s[1])), p[0], p[1]);
        return (channels > 2 ? p[0] : s[0]) + (channels > 3 ? p[1] : s[1]);
    };
#pragma unroll 1
    for (int t = end - 1; t >= first; --t) {
        Entries h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const ulonglong2 v = ck[e * threads];
            h[e][0] = v.x;
            h[e][1] = v.y;
        }
#pragma unroll 1
        for (int i = first; i < t; ++i) at.advance(i, A, h);
        const Operands o = at.operands(t);
        const f32x2 d[2] = {pk(o.d.x, o.d.y), pk(o.d.z, o.d.w)}, x[2] = {pk(o.x.x, o.x.y), pk(o.x.z, o.x.w)},
                    g[2] = {pk(o.g.x, o.g.y), pk(o.g.z, o.g.w)};
        const float B[4] = {o.B.x, o.B.y, o.B.z, o.B.w}, C[4] = {o.C.x, o.C.y, o.C.z, o.C.w};
        f32x2 y[2] = {0ull, 0ull}, sb[2] = {0ull, 0ull}, sa[2] = {0ull, 0ull};
        float vB[4], vC[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f32x2 lam[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x2 w = exp2_2(mul2(d[j], A[e][j])), wh = mul2(w, h[e][j]);
                h[e][j] = fma2(x[j], pk(B[e], B[e]), wh);
                y[j] = entry(e, pk(C[e], C[e]), h[e][j], y[j]);
                lam[j] = fma2(g[j], pk(C[e], C[e]), m[e][j]);
                sb[j] = entry(e, lam[j], pk(B[e], B[e]), sb[j]);
                m[e][j] = mul2(lam[j], w);
                const f32x2 held = mul2(lam[j], wh);
                dA[e][j] = fma2(held, d[j], dA[e][j]);
                sa[j] = entry(e, held, A[e][j], sa[j]);
            }
            vC[e] = over_channels(h[e], g);
            vB[e] = over_channels(lam, x);
        }
        float* row = red + t % kRun * 2 * Lane<LP>::NP;
        join_lanes<LP>(y[0], y[1], lane, y_row + t * at.cc);
        join_warp<LP>(vC, lane, row + Lane<LP>::NP);
        join_lanes<LP>(sb[0], sb[1], lane, at.s_x + t * at.cc + 4 * at.qd);
        join_lanes<LP>(sa[0], sa[1], lane, at.s_g + t * at.cc + 4 * at.qd);
        join_warp<LP>(vB, lane, row);
    }
}

// PAD: the lanes hold more entries than there are, or the blocks more channels, or the runs more tokens (`alone`).
template <typename T, int LP, int BLOCK, bool PAD>
__global__ void __launch_bounds__(128, 2) selective_block_kernel(SelectiveArgs a, const T* __restrict__ dy, int nblocks,
                                                                 const float* start, const float* end, float* dA_parts,
                                                                 T* __restrict__ dx, T* __restrict__ ddt,
                                                                 T* __restrict__ dz, float* __restrict__ dbc,
                                                                 float* __restrict__ chan, bool vec, bool vecb) {
    using K = Blk<LP, BLOCK>;
    constexpr int NP = K::NP;
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = threads / 32;
    const int cc = K::channels(threads), N = a.dstate, k = blockIdx.y;
    const Rows<T> r = rows_at<T, BLOCK>(a, dy, cc);
    const int qd = tid / LP, q = tid % LP, mine = r.nc - 4 * qd;
    const int64_t c = r.c0 + 4 * qd, n = (int64_t)a.channels * N, row = ((int64_t)r.b * nblocks + k) * n;
    float *s_d = sm, *s_x = s_d + BLOCK * cc, *s_g = s_x + BLOCK * cc, *s_y = s_g + BLOCK * cc, *s_B = s_y + BLOCK * cc,
          *s_C = s_B + BLOCK * NP, *s_red = s_C + BLOCK * NP;
    ulonglong2* ck = reinterpret_cast<ulonglong2*>(s_red + warps * kRun * 2 * NP) + tid;
    float unused[4];
    const float undefined = stage_block<T, LP, BLOCK>(a, r, s_d, s_x, s_g, s_B, s_C, vec, vecb, unused);
    Entries A, h, m, dA;
    read_entries(a.A, c, mine, N, 4 * q, kLog2e, A);
    grid_dep_wait();  // the hops
    read_entries(start + row, c, start != nullptr ? mine : 0, N, 4 * q, 1.f, h);
    read_entries(end + row, c, end != nullptr ? mine : 0, N, 4 * q, 1.f, m);
#pragma unroll
    for (int e = 0; e < 4; ++e) dA[e][0] = dA[e][1] = 0ull;
    bool finite = true;
    if (PAD) finite = __syncthreads_or(undefined != 0.f) == 0;
    else __syncthreads();
    const int steps = max(0, r.last - r.tb), runs = (steps + kRun - 1) / kRun;  // tokens past the length change nothing

    const Lane<LP> at = {s_d, s_x, s_g, s_B, s_C, cc, qd, q};
    auto advance = [&](int t) { at.advance(t, A, h); };
    auto operands = [&](int t) { return at.operands(t); };
    auto join = [&](f32x2 lo, f32x2 hi, float* to) { join_lanes<LP>(lo, hi, lane, to + 4 * qd); };
    // four values over the warp's channels, to entries 4 q .. of a token's row of dB (half = 0) or dC (1); join_warp written
    // out, which keeps this kernel's registers as they are without `alone` (500 us at 2 x 4096 x 2048 x 16, 507 otherwise)
    auto join_channels = [&](float (&v)[4], int t, int half) {
        constexpr int CW = 32 / LP, LEFT = CW >= 4 ? 1 : 4 / CW;
        int which = 0;
        fold_between<4, 16, LP>(v, lane, which);
        float* to = s_red + ((warp * kRun + t % kRun) * 2 + half) * NP + 4 * q + which;
        if (CW <= 4 || ((lane / LP) & (CW / 4 > 0 ? CW / 4 - 1 : 0)) == 0) {
#pragma unroll
            for (int e = 0; e < LEFT; ++e) to[e] = v[e];
        }
    };
    // tokens t0 .. t0 + 3 from the states before them: forward with y and dC, then backward with the rest
    auto half = [&](int t0) {
        f32x2 w[kHeld][4][2], wh[kHeld][4][2];  // the decays, and the decayed states
        Operands o = operands(t0);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int t = t0 + i;
            const Operands next = operands(i + 1 < kHeld ? t + 1 : t);
            const f32x2 d[2] = {pk(o.d.x, o.d.y), pk(o.d.z, o.d.w)}, x[2] = {pk(o.x.x, o.x.y), pk(o.x.z, o.x.w)},
                        g[2] = {pk(o.g.x, o.g.y), pk(o.g.z, o.g.w)};
            const float B[4] = {o.B.x, o.B.y, o.B.z, o.B.w}, C[4] = {o.C.x, o.C.y, o.C.z, o.C.w};
            f32x2 y[2];
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    w[i][e][j] = exp2_2(mul2(d[j], A[e][j]));
                    wh[i][e][j] = mul2(w[i][e][j], h[e][j]);
                    h[e][j] = fma2(x[j], pk(B[e], B[e]), wh[i][e][j]);
                    y[j] = e == 0 ? mul2(pk(C[0], C[0]), h[0][j]) : fma2(pk(C[e], C[e]), h[e][j], y[j]);
                }
                v[e] = sum2(fma2(h[e][1], g[1], mul2(h[e][0], g[0])));
            }
            join(y[0], y[1], s_y + t * cc);
            join_channels(v, t, 1);
            o = next;
        }
#pragma unroll
        for (int i = kHeld - 1; i >= 0; --i) {
            const int t = t0 + i;
            const Operands next = operands(i > 0 ? t - 1 : t);
            const f32x2 d[2] = {pk(o.d.x, o.d.y), pk(o.d.z, o.d.w)}, x[2] = {pk(o.x.x, o.x.y), pk(o.x.z, o.x.w)},
                        g[2] = {pk(o.g.x, o.g.y), pk(o.g.z, o.g.w)};
            const float B[4] = {o.B.x, o.B.y, o.B.z, o.B.w}, C[4] = {o.C.x, o.C.y, o.C.z, o.C.w};
            f32x2 sb[2], sa[2];
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f32x2 lam[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    lam[j] = fma2(g[j], pk(C[e], C[e]), m[e][j]);
                    sb[j] = e == 0 ? mul2(lam[j], pk(B[0], B[0])) : fma2(lam[j], pk(B[e], B[e]), sb[j]);
                    m[e][j] = mul2(lam[j], w[i][e][j]);
                    const f32x2 held = mul2(lam[j], wh[i][e][j]);
                    dA[e][j] = fma2(held, d[j], dA[e][j]);
                    sa[j] = e == 0 ? mul2(held, A[0][j]) : fma2(held, A[e][j], sa[j]);
                }
                v[e] = sum2(fma2(lam[1], x[1], mul2(lam[0], x[0])));
            }
            // in place of dt x and g: every lane of these channels, lanes of one warp, has read the token's
            join(sb[0], sb[1], s_x + t * cc);
            join(sa[0], sa[1], s_g + t * cc);
            join_channels(v, t, 0);
            o = next;
        }
    };

    // forward: a checkpoint before every run
    for (int j = 0; j < runs; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) ck[(4 * j + e) * threads] = make_ulonglong2(h[e][0], h[e][1]);
        if (j + 1 < runs) {
#pragma unroll 2
            for (int i = 0; i < kRun; ++i) advance(j * kRun + i);
        }
    }
    auto restore = [&](int j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const ulonglong2 v = ck[(4 * j + e) * threads];
            h[e][0] = v.x;
            h[e][1] = v.y;
        }
    };
    // backward, run by run, its second half first
    const int64_t place = ((int64_t)r.tile * a.batch + r.b) * a.seqlen;  // dbc: (tiles, batch, seqlen, ngroups, 2, dstate)
    // whether the states after the last run's tokens (none was infinite before if these are finite) and the gradient that comes
    // to it are finite, so that its tokens past the length do add zeros
    auto settled = [&](int j) {
        restore(j);
#pragma unroll 1
        for (int t = j * kRun; t < steps; ++t) advance(t);
        float undefined = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float lo, hi;
                unpk(fma2(h[e][i], 0ull, mul2(m[e][i], 0ull)), lo, hi);
                undefined += lo + hi;
            }
        return __syncthreads_or(undefined != 0.f) == 0;
    };
    auto store_run = [&](int j) {
        __syncthreads();
        for (int i = tid; i < kRun * 2 * LP; i += threads) {  // four entries of a token's dB or dC, over the warps
            const int tt = i / (2 * LP), which = i / LP % 2, e = i % LP * 4, t = r.tb + j * kRun + tt;
            float4 s = *reinterpret_cast<const float4*>(s_red + 4 * i);
            for (int w = 1; w < warps; ++w) {
                const float4 u = *reinterpret_cast<const float4*>(s_red + w * kRun * 2 * NP + 4 * i);
                s = make_float4(s.x + u.x, s.y + u.y, s.z + u.z, s.w + u.w);
            }
            const float o[4] = {s.x, s.y, s.z, s.w};
            store_vec<float, 4>(dbc + (((place + t) * a.ngroups + r.grp) * 2 + which) * N + e,
                                !PAD || t < r.last ? Vec<float, 4>::of(o) : Vec<float, 4>::zero(), t < r.te ? N - e : 0,
                                N % 4 == 0);
        }
        __syncthreads();
    };
    int j = runs - 1;
    if constexpr (PAD) {
        const bool careful = !finite || (steps % kRun != 0 && !settled(j));
        for (; careful && j >= 0; --j) {
            alone<LP>(at, ck + 4 * j * threads, j * kRun, min(steps, (j + 1) * kRun), N - 4 * q, mine, s_y + 4 * qd,
                      s_red + warp * kRun * 2 * NP + 4 * q, A, m, dA);
            store_run(j);
        }
    }
    for (; j >= 0; --j) {
#pragma unroll 1
        for (int s = 1; s >= 0; --s) {
            restore(j);
            if (s == 1) {
#pragma unroll 2
                for (int i = 0; i < kHeld; ++i) advance(j * kRun + i);
            }
            half(j * kRun + s * kHeld);
        }
        store_run(j);
    }
    // tokens past the last run have no gradient in B and C
    for (int i = tid; i < (r.te - r.tb - runs * kRun) * 2 * N; i += threads) {
        const int t = r.tb + runs * kRun + i / (2 * N);
        dbc[((place + t) * a.ngroups + r.grp) * 2 * N + i % (2 * N)] = 0.f;
    }
    write_entries(dA_parts + row, c, mine, N, 4 * q, dA);  // in place of the start state, where that came from a hop
    __syncthreads();

    // per token and channel
    const int v0 = tid % (cc / 4), w0 = tid / (cc / 4), vc = r.nc - 4 * v0;
    constexpr int M = K::CONVS < 2 ? K::CONVS : 2;
    float dD[4] = {0.f, 0.f, 0.f, 0.f}, dbias[4] = {0.f, 0.f, 0.f, 0.f}, bias[4], Dc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        bias[e] = a.dto.bias != nullptr && e < vc ? a.dto.bias[r.c0 + 4 * v0 + e] : 0.f;
        Dc[e] = a.D != nullptr && e < vc ? a.D[r.c0 + 4 * v0 + e] : 0.f;
    }
    const bool gated = r.z != nullptr;
#pragma unroll 1
    for (int i0 = 0; i0 < K::CONVS; i0 += M) {
        const int t0 = w0 + i0 * K::CONV;
        const Loaded<T, M> l = load_rows<T, M, K::CONV>(a, r, r.tb + t0, v0, vec);
        float raw[4 * M], slope[4 * M], g[4 * M], fz[4 * M];
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                raw[4 * i + e] = l.d[i].get(e) + bias[e];
                slope[4 * i + e] = 1.f;
                g[4 * i + e] = l.dy[i].get(e);
                fz[4 * i + e] = 0.f;
            }
        if (a.dto.softplus) {
#pragma unroll
            for (int i = 0; i < 4 * M; ++i) slope[i] = sigmoid(raw[i]);
        }
        if (a.dto.limit) {
#pragma unroll
            for (int i = 0; i < 4 * M; ++i) {
                const float s = a.dto.softplus ? softplus(raw[i]) : raw[i];
                slope[i] = (s >= a.dto.lo && s <= a.dto.hi) ? slope[i] : 0.f;
            }
        }
        if (gated) {
#pragma unroll
            for (int i = 0; i < M; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float zv = l.z[i].get(e), sg = sigmoid(zv);
                    const int t = t0 + i * K::CONV < BLOCK ? t0 + i * K::CONV : 0;
                    fz[4 * i + e] = g[4 * i + e] * fmaf(Dc[e], l.x[i].get(e), s_y[t * cc + 4 * v0 + e]) * sg * fmaf(zv, 1.f - sg, 1.f);
                    g[4 * i + e] *= zv * sg;
                }
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int t = t0 + i * K::CONV;
            if (K::CONV * K::CONVS != BLOCK && t >= BLOCK) break;
            const bool live = r.tb + t < r.last;
            const float4 d4 = *reinterpret_cast<const float4*>(s_d + t * cc + 4 * v0);
            const float4 b4 = *reinterpret_cast<const float4*>(s_x + t * cc + 4 * v0);
            const float4 a4 = *reinterpret_cast<const float4*>(s_g + t * cc + 4 * v0);
            const float dt[4] = {d4.x, d4.y, d4.z, d4.w}, sb[4] = {b4.x, b4.y, b4.z, b4.w}, sa[4] = {a4.x, a4.y, a4.z, a4.w};
            float ox[4], od[4], oz[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float xv = l.x[i].get(e);
                ox[e] = live ? fmaf(dt[e], sb[e], Dc[e] * g[4 * i + e]) : 0.f;
                od[e] = live ? fmaf(xv, sb[e], kLn2 * sa[e]) * slope[4 * i + e] : 0.f;
                oz[e] = live ? fz[4 * i + e] : 0.f;
                dD[e] += live ? g[4 * i + e] * xv : 0.f;
                dbias[e] += od[e];
            }
            const int64_t o = ((int64_t)r.b * a.seqlen + r.tb + t) * a.channels + r.c0 + 4 * v0;
            const int valid = r.tb + t < r.te ? vc : 0;
            store_vec<T, 4>(dx + o, Vec<T, 4>::of(ox), valid, vec);
            store_vec<T, 4>(ddt + o, Vec<T, 4>::of(od), valid, vec);
            if (gated) store_vec<T, 4>(dz + o, Vec<T, 4>::of(oz), valid, vec);
        }
    }
    __syncthreads();
    float* sums = sm + w0 * 2 * cc + 4 * v0;
    *reinterpret_cast<float4*>(sums) = make_float4(dD[0], dD[1], dD[2], dD[3]);
    *reinterpret_cast<float4*>(sums + cc) = make_float4(dbias[0], dbias[1], dbias[2], dbias[3]);
    __syncthreads();
    for (int i = tid; i < 2 * cc; i += threads) {
        if (i % cc >= r.nc) continue;
        float s = 0.f;
        for (int w = 0; w < K::CONV; ++w) s += sm[w * 2 * cc + i];
        chan[(((int64_t)r.b * nblocks + k) * 2 + i / cc) * a.channels + r.c0 + i % cc] = s;
    }
}

template <typename T, int LP, int BLOCK>
int backward_blocks(const SelectiveArgs& a, const SelectiveParts& p, const SelectiveGrads& g, float* ws, cudaStream_t s) {
    using K = Blk<LP, BLOCK>;
    float *hops = ws, *mus = hops + p.hops, *nu0 = mus + p.hops, *dtsum = nu0 + p.nu0, *chan = dtsum + p.dtsum,
          *dbc = chan + p.chan;
    const T* dy = static_cast<const T*>(g.dy);
    const bool vec = rows_of_four(a, g.dx, g.ddt, sizeof(T)) && aligned_to(g.dy, 4 * sizeof(T)) &&
                     aligned_to(g.dz, 4 * sizeof(T)) && a.channels % 4 == 0;
    const bool vecb = states_of_four(a, sizeof(T));
    const int threads = selective_block_threads(a), smem = K::floats(threads) * 4, smem_terms = K::floats_terms(threads) * 4;
    const int most = LP == 2 ? 64 : 128;
    const dim3 grid(a.ngroups * p.tiles, p.nblocks, a.batch);
    int r = ensure_smem_limit(reinterpret_cast<const void*>(selective_terms_kernel<T, LP, BLOCK>), K::floats_terms(most) * 4);
    const bool pad = a.dstate < K::NP || a.channels / a.ngroups % K::channels(threads) != 0 || a.seqlen % kRun != 0 || a.lengths != nullptr;
    const auto block = pad ? selective_block_kernel<T, LP, BLOCK, true> : selective_block_kernel<T, LP, BLOCK, false>;
    if (r == SSD_OK) r = ensure_smem_limit(reinterpret_cast<const void*>(block), K::floats(most) * 4);
    if (r != SSD_OK) return r;
    T *dx = static_cast<T*>(g.dx), *ddt = static_cast<T*>(g.ddt), *dz = static_cast<T*>(g.dz);
    if (p.nblocks == 1 && g.dinit == nullptr) {  // the block starts and ends with the row
        launch_begin(kKindSelectiveBwd, s);
        block<<<grid, threads, smem, s>>>(a, dy, 1, a.init, g.dfinal, hops, dx, ddt, dz, dbc, chan, vec, vecb);
        r = launch_end(kKindSelectiveBwd, s);
    } else {
        launch_begin(kKindSelectiveBwd, s);
        selective_terms_kernel<T, LP, BLOCK><<<grid, threads, smem_terms, s>>>(a, dy, p.nblocks, hops, mus, nu0, dtsum, vec, vecb);
        r = launch_end(kKindSelectiveBwd, s);
        if (r != SSD_OK) return r;
        r = launch_selective_hops(a, g, p, hops, mus, nu0, dtsum, s);
        if (r != SSD_OK) return r;
        launch_begin(kKindSelectiveBwd, s);
        if (pad)
            launch_dependent(selective_block_kernel<T, LP, BLOCK, true>, grid, dim3(threads), smem, s, a, dy, p.nblocks, hops, mus, hops,
                             dx, ddt, dz, dbc, chan, vec, vecb);
        else
            launch_dependent(selective_block_kernel<T, LP, BLOCK, false>, grid, dim3(threads), smem, s, a, dy, p.nblocks, hops, mus,
                             hops, dx, ddt, dz, dbc, chan, vec, vecb);
        r = launch_end(kKindSelectiveBwd, s);
    }
    if (r != SSD_OK) return r;
    return launch_selective_sums(a, g, p, hops, chan, dbc, s);
}

template <typename T, int LP>
int backward_lanes(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s) {
    const SelectiveParts p = selective_parts(a);
    if constexpr (LP <= 16)
        if (p.tokens == 16) return backward_blocks<T, LP, 16>(a, p, g, ws, s);
    return backward_blocks<T, LP, 32>(a, p, g, ws, s);
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
}  // namespace ssd
