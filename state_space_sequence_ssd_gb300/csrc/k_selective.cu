// k_selective.cu -- the selective scan with one decay per channel and state entry, forward.  Per row b, channel c
// (group g = c / (channels / ngroups)) and token t:
//
//   h[n] <- exp(dt[t][c] A[c][n]) h[n] + dt[t][c] x[t][c] B[t][g][n]
//   y[t][c] = sum_n C[t][g][n] h[n] + D[c] x[t][c],   then y <- y z sigmoid(z) with a gate
//
// What it costs: one exponential and four multiply-adds or multiplies per (token, channel, state entry).  The
// special function units give 32 exponentials and the float32 units 128 results per clock and SM, so both need four
// clocks for a warp's 32 entries, and the units, not HBM, set the floor (the exponentials alone: 57 us at
// 2 x 4096 tokens x 4096 channels x 16 entries, whose bytes take 40 us).
//
// Layout: a lane holds four state entries of one channel, so the four chains of the recurrence and the exponentials
// of the next tokens (which wait for nothing) fill the pipelines with few warps, and 128 bits of B or C feed four
// entries.  A block of four warps covers 4 * 32 / LP channels of one group; the tokens' dt and dt x are staged once
// per channel in shared memory, twice each, as the packed pairs that the arithmetic takes, and B and C as float32.
// A tile's loads are in registers while the tile before it is computed.  The sum over a channel's lanes is taken
// for four tokens at a time, each lane ending with one of them.
//
// With few channels the sequence is split into chunks: the same kernel first computes each chunk's own end state
// from zero, a hop carries the states across the chunks (the decay over a chunk is exp(A sum dt)), and the second
// run starts every chunk from its true state.  That costs the exponentials twice, so it is used only where one run
// would leave SMs idle.
#include "selective.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;

template <int LP>
struct Tile {
    static constexpr int CW = 32 / LP;          // channels of a warp
    static constexpr int CC = kWarps * CW;      // channels of a block
    static constexpr int N4 = 4 * LP;           // state entries, padded
    static constexpr int TS = LP <= 8 ? 32 : LP == 16 ? 16 : 8;  // tokens of a tile
    static constexpr int CV = CC / 4;           // vectors of four channels per token
    static constexpr int XI = (TS * CV + kThreads - 1) / kThreads;   // such vectors per thread
    static constexpr int BI = TS * LP / kThreads > 0 ? TS * LP / kThreads : 1;  // vectors of B (and of C) per thread
    static constexpr int RB = LP < 4 ? LP : 4;  // tokens whose sums are folded together
};

template <typename T, int LP, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads) selective_kernel(SelectiveArgs a, int chunk, int nchunks, T* __restrict__ y,
                                                             float* __restrict__ final_state, float* __restrict__ hops,
                                                             float* __restrict__ dtsum, bool vec, bool vecb) {
    using K = Tile<LP>;
    constexpr int TS = K::TS, CC = K::CC, CV = K::CV;
    __shared__ float4 s_dt[TS * CC];  // (dt, dt, dt x, dt x), swizzled by channel
    __shared__ float4 s_B[TS * LP];
    __shared__ float4 s_C[STATE_ONLY ? 1 : TS * LP];
    __shared__ float s_y[STATE_ONLY ? 1 : TS * CC];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = a.channels / a.ngroups, tiles = (per + CC - 1) / CC;
    const int grp = blockIdx.x / tiles, g0 = grp * per, cb = (blockIdx.x % tiles) * CC;  // channels cb.. of the group
    const int b = blockIdx.z, part = blockIdx.y, N = a.dstate;
    const int len = row_length(a.lengths, b, a.seqlen);
    const int tb = part * chunk, te = min(tb + chunk, a.seqlen);
    const T* xp = static_cast<const T*>(a.x) + b * a.x_batch + g0 + cb;
    const T* dp = static_cast<const T*>(a.dt) + b * a.dt_batch + g0 + cb;
    const T* zp = a.z == nullptr ? nullptr : static_cast<const T*>(a.z) + b * a.z_batch + g0 + cb;
    const T* Bp = static_cast<const T*>(a.B) + b * a.B_batch + (int64_t)grp * N;
    const T* Cp = static_cast<const T*>(a.C) + b * a.C_batch + (int64_t)grp * N;
    const int nc = min(CC, per - cb);  // channels of this block

    // this lane's channel and four state entries
    const int cl = warp * K::CW + lane / LP, q = lane % LP;
    const bool mine = cl < nc;
    const int64_t ci = g0 + cb + cl;
    const int nvalid = mine ? max(0, min(4, N - 4 * q)) : 0;
    f32x2 A01, A23, h01, h23;
    {
        const Vec<float, 4> A4 = load_vec<float, 4>(a.A + (mine ? ci * N + 4 * q : 0), nvalid, false);
        A01 = pk(A4.get(0) * kLog2e, A4.get(1) * kLog2e);
        A23 = pk(A4.get(2) * kLog2e, A4.get(3) * kLog2e);
        h01 = h23 = 0ull;
        const float* from = nullptr;
        if (!STATE_ONLY && nchunks > 1) from = hops + ((int64_t)b * nchunks + part) * a.channels * N;
        else if (!STATE_ONLY && a.init != nullptr) from = a.init + (int64_t)b * a.channels * N;
        if (from != nullptr) {
            const Vec<float, 4> h4 = load_vec<float, 4>(from + (mine ? ci * N + 4 * q : 0), nvalid, false);
            h01 = pk(h4.get(0), h4.get(1));
            h23 = pk(h4.get(2), h4.get(3));
        }
    }
    float bias[4] = {0.f, 0.f, 0.f, 0.f}, Dv[4] = {0.f, 0.f, 0.f, 0.f}, dsum[4] = {0.f, 0.f, 0.f, 0.f};
    const int v0 = tid % CV;  // every staged vector of this thread is of the same four channels
    static_assert(kThreads % CV == 0, "a thread's vectors share their channels");
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (4 * v0 + e < nc) {
            if (a.dto.bias != nullptr) bias[e] = a.dto.bias[g0 + cb + 4 * v0 + e];
            if (a.D != nullptr) Dv[e] = a.D[g0 + cb + 4 * v0 + e];
        }

    Vec<T, 4> rx[K::XI], rd[K::XI], rz[K::XI], rB[K::BI], rC[K::BI];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < K::XI; ++i) {
            const int idx = tid + i * kThreads, t = t0 + idx / CV;
            const int valid = (idx < TS * CV && t < len && t < te) ? max(0, nc - 4 * v0) : 0;
            rx[i] = load_vec<T, 4>(xp + t * a.x_token + 4 * v0, valid, vec);
            rd[i] = load_vec<T, 4>(dp + t * a.dt_token + 4 * v0, valid, vec);
            if (!STATE_ONLY && zp != nullptr) rz[i] = load_vec<T, 4>(zp + t * a.z_token + 4 * v0, valid, vec);
        }
#pragma unroll
        for (int i = 0; i < K::BI; ++i) {
            const int idx = tid + i * kThreads, t = t0 + idx / LP, n = 4 * (idx % LP);
            const int valid = (idx < TS * LP && t < len && t < te) ? max(0, N - n) : 0;
            rB[i] = load_vec<T, 4>(Bp + t * a.B_token + n, valid, vecb);
            if (!STATE_ONLY) rC[i] = load_vec<T, 4>(Cp + t * a.C_token + n, valid, vecb);
        }
    };
    fetch(tb);
    for (int t0 = tb; t0 < te; t0 += TS) {
        if (STATE_ONLY && t0 >= len) break;
        Vec<T, 4> cx[K::XI], cz[K::XI];  // this tile's x and z, for its outputs
#pragma unroll
        for (int i = 0; i < K::XI; ++i) {
            const int idx = tid + i * kThreads;
            if (idx < TS * CV) {
                const bool live = t0 + idx / CV < len && t0 + idx / CV < te;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // a token past the length keeps the state: dt = 0
                    const float d = live ? effective(rd[i].get(e), bias[e], a.dto) : 0.f;
                    const float dx = d * rx[i].get(e);
                    s_dt[(idx / CV) * CC + 4 * v0 + (e ^ ((v0 >> 1) & 3))] = make_float4(d, d, dx, dx);
                    if (STATE_ONLY) dsum[e] += d;
                }
            }
            cx[i] = rx[i];
            if (!STATE_ONLY) cz[i] = rz[i];
        }
#pragma unroll
        for (int i = 0; i < K::BI; ++i) {
            const int idx = tid + i * kThreads;
            if (idx < TS * LP) {
                s_B[idx] = make_float4(rB[i].get(0), rB[i].get(1), rB[i].get(2), rB[i].get(3));
                if (!STATE_ONLY)
                    s_C[idx] = make_float4(rC[i].get(0), rC[i].get(1), rC[i].get(2), rC[i].get(3));
            }
        }
        __syncthreads();
        if (t0 + TS < te) fetch(t0 + TS);
        const int steps = min(TS, min(te, len) - t0);  // at most; none for a tile past the length
        const float4* sd = s_dt + ((cl & ~3) | ((cl & 3) ^ ((cl >> 3) & 3)));
#pragma unroll 2
        for (int j = 0; j < steps; j += K::RB) {
            float acc[K::RB];
#pragma unroll
            for (int i = 0; i < K::RB; ++i) {
                const float4 d = sd[(j + i) * CC];
                const float4 Bq = s_B[(j + i) * LP + q];
                const f32x2 dd = pk(d.x, d.y), dx = pk(d.z, d.w);
                const f32x2 a01 = exp2_2(mul2(dd, A01)), a23 = exp2_2(mul2(dd, A23));
                h01 = fma2(a01, h01, mul2(dx, pk(Bq.x, Bq.y)));
                h23 = fma2(a23, h23, mul2(dx, pk(Bq.z, Bq.w)));
                if (!STATE_ONLY) {
                    const float4 Cq = s_C[(j + i) * LP + q];
                    acc[i] = sum2(fma2(pk(Cq.z, Cq.w), h23, mul2(pk(Cq.x, Cq.y), h01)));
                }
            }
            if (!STATE_ONLY) {
                int which = 0;
                const float s = fold_lanes<K::RB, LP / 2>(acc, q, which);
                if (q % (LP / K::RB) == 0) s_y[(j + which) * CC + cl] = s;
            }
        }
        __syncthreads();
        if (!STATE_ONLY) {
#pragma unroll
            for (int i = 0; i < K::XI; ++i) {
                const int idx = tid + i * kThreads, t = t0 + idx / CV, valid = nc - 4 * v0;
                if (idx >= TS * CV || t >= te || valid <= 0) continue;
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = 0.f;
                    if (t < len) {
                        v = fmaf(Dv[e], cx[i].get(e), s_y[(idx / CV) * CC + 4 * v0 + e]);
                        if (zp != nullptr) {
                            const float zv = cz[i].get(e);
                            v *= zv * sigmoid(zv);
                        }
                    }
                    o[e] = v;
                }
                store_vec<T, 4>(y + ((int64_t)b * a.seqlen + t) * a.channels + g0 + cb + 4 * v0, Vec<T, 4>::of(o), valid, vec);
            }
        }
    }
    float* to = nullptr;
    if (STATE_ONLY) to = hops + ((int64_t)b * nchunks + part + 1) * a.channels * N;  // carried into the next chunk
    else if (final_state != nullptr && te == a.seqlen) to = final_state + (int64_t)b * a.channels * N;
    if (to != nullptr && mine) {
        float h4[4];
        unpk(h01, h4[0], h4[1]);
        unpk(h23, h4[2], h4[3]);
        store_vec<float, 4>(to + ci * N + 4 * q, Vec<float, 4>::of(h4), nvalid, N % 4 == 0 && (reinterpret_cast<uintptr_t>(to) & 15) == 0);
    }
    if (STATE_ONLY) {
        // sum of dt over the chunk, per channel: the threads of one vector's tokens, in shared memory
        __syncthreads();
        float* buf = reinterpret_cast<float*>(s_dt);
#pragma unroll
        for (int e = 0; e < 4; ++e) buf[(tid / CV) * CC + 4 * v0 + e] = dsum[e];
        __syncthreads();
        for (int c = tid; c < nc; c += kThreads) {
            float s = 0.f;
            for (int r = 0; r < kThreads / CV; ++r) s += buf[r * CC + c];
            dtsum[((int64_t)b * nchunks + part) * a.channels + g0 + cb + c] = s;
        }
    }
}

// The states that every chunk starts from: hops[0] = init, hops[k + 1] = exp(A dtsum[k]) hops[k] + (chunk k's own end
// state, which hops[k + 1] holds on entry).
__global__ void __launch_bounds__(256) selective_hop_kernel(const float* __restrict__ A, const float* __restrict__ init,
                                                            int channels, int dstate, int nchunks, float* __restrict__ hops,
                                                            const float* __restrict__ dtsum) {
    const int64_t n = (int64_t)channels * dstate, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int b = blockIdx.y;
    if (i >= n) return;
    const float A2 = A[i] * kLog2e;
    float h = init != nullptr ? init[b * n + i] : 0.f;
    float* hp = hops + b * n * nchunks + i;
    const float* dp = dtsum + (int64_t)b * nchunks * channels + i / dstate;
    hp[0] = h;
#pragma unroll 4
    for (int k = 0; k + 1 < nchunks; ++k) {
        h = fmaf(exp2_fast(A2 * dp[(int64_t)k * channels]), h, hp[(k + 1) * n]);
        hp[(k + 1) * n] = h;
    }
}

template <typename T, int LP>
int forward_lanes(const SelectiveArgs& a, int chunks, T* y, float* final_state, float* ws, cudaStream_t s) {
    using K = Tile<LP>;
    const int per = a.channels / a.ngroups, tiles = a.ngroups * ceil_div(per, K::CC);
    const int chunk = ceil_div(ceil_div(a.seqlen, chunks), K::TS) * K::TS;
    const int nchunks = ceil_div(a.seqlen, chunk);
    const bool vec = rows_of_four(a, y, nullptr, sizeof(T)), vecb = states_of_four(a, sizeof(T));
    float* hops = ws;
    float* dtsum = ws == nullptr ? nullptr : ws + (int64_t)a.batch * nchunks * a.channels * a.dstate;
    int r = SSD_OK;
    if (nchunks > 1) {
        launch_begin(kKindSelective, s);
        selective_kernel<T, LP, true><<<dim3(tiles, nchunks - 1, a.batch), kThreads, 0, s>>>(a, chunk, nchunks, y, nullptr, hops,
                                                                                          dtsum, vec, vecb);
        r = launch_end(kKindSelective, s);
        if (r != SSD_OK) return r;
        launch_begin(kKindSelective, s);
        selective_hop_kernel<<<dim3((unsigned)ceil_div64((int64_t)a.channels * a.dstate, 256), a.batch), 256, 0, s>>>(
            a.A, a.init, a.channels, a.dstate, nchunks, hops, dtsum);
        r = launch_end(kKindSelective, s);
        if (r != SSD_OK) return r;
    }
    launch_begin(kKindSelective, s);
    selective_kernel<T, LP, false><<<dim3(tiles, nchunks, a.batch), kThreads, 0, s>>>(a, chunk, nchunks, y, final_state, hops,
                                                                                   dtsum, vec, vecb);
    return launch_end(kKindSelective, s);
}

template <typename T>
int forward_of(const SelectiveArgs& a, int chunks, void* y, float* final_state, float* ws, cudaStream_t s) {
    T* yt = static_cast<T*>(y);
    switch (selective_lanes(a.dstate)) {
        case 2: return forward_lanes<T, 2>(a, chunks, yt, final_state, ws, s);
        case 4: return forward_lanes<T, 4>(a, chunks, yt, final_state, ws, s);
        case 8: return forward_lanes<T, 8>(a, chunks, yt, final_state, ws, s);
        case 16: return forward_lanes<T, 16>(a, chunks, yt, final_state, ws, s);
        case 32: return forward_lanes<T, 32>(a, chunks, yt, final_state, ws, s);
        default: return SSD_ERR_UNSUPPORTED;
    }
}

// ------------------------------------------------------------------------------------------------ one token
// A lane holds four state entries of one channel for R rows, and LP lanes share the channel.  Bound by HBM: the state
// is read and written once.  The rows' states are loaded together and A once for them; each of the first R lanes
// forms one row's dt and gate for the others, and ends with that row's output.  An idle row (slot -1) writes zeros
// and leaves every slot alone.
template <typename T, int LP, int R>
__global__ void __launch_bounds__(256) selective_step_kernel(SelectiveArgs a, float* __restrict__ state,
                                                             const int* __restrict__ slots, int nslots, T* __restrict__ y,
                                                             int* err, bool vecs, bool vecb) {
    const int b0 = blockIdx.y * R, N = a.dstate, q = threadIdx.x % LP;
    const int64_t c = (int64_t)blockIdx.x * (256 / LP) + threadIdx.x / LP;
    const bool mine = c < a.channels;
    const int nvalid = mine ? max(0, min(4, N - 4 * q)) : 0;
    const int g = mine ? (int)(c / (a.channels / a.ngroups)) : 0;
    int slot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) slot[r] = b0 + r < a.batch ? row_slot(slots, b0 + r, nslots, err) : -1;
    Vec<float, 4> h[R];
    Vec<T, 4> Bv[R], Cv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int got = slot[r] >= 0 ? nvalid : 0;
        h[r] = load_vec<float, 4, true>(state + ((int64_t)slot[r] * a.channels + c) * N + 4 * q, got, vecs);
        const int64_t bc = (int64_t)g * N + 4 * q;
        Bv[r] = load_vec<T, 4>(static_cast<const T*>(a.B) + (b0 + r) * a.B_batch + bc, got, vecb);
        Cv[r] = load_vec<T, 4>(static_cast<const T*>(a.C) + (b0 + r) * a.C_batch + bc, got, vecb);
    }
    // lane q: row b0 + q's scalars
    const bool own = mine && q < R && b0 + q < a.batch;
    float xq = 0.f, dq = 0.f, zq = 0.f, Dq = 0.f;
    if (own) {
        xq = to_f32<T>(static_cast<const T*>(a.x)[(b0 + q) * a.x_batch + c]);
        dq = to_f32<T>(static_cast<const T*>(a.dt)[(b0 + q) * a.dt_batch + c]);
        if (a.z != nullptr) zq = to_f32<T>(static_cast<const T*>(a.z)[(b0 + q) * a.z_batch + c]);
        if (a.D != nullptr) Dq = __ldg(a.D + c);
    }
    const float bias = a.dto.bias != nullptr && mine ? __ldg(a.dto.bias + c) : 0.f;
    const Vec<float, 4> A4 = load_vec<float, 4>(a.A + (mine ? c * N + 4 * q : 0), nvalid, vecs);
    const f32x2 log2e = pk(kLog2e, kLog2e), A01 = mul2(A4.pair(0), log2e), A23 = mul2(A4.pair(1), log2e);
    dq = effective(dq, bias, a.dto);
    const float dxq = dq * xq;
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float d = __shfl_sync(0xffffffffu, dq, r, LP), dx = __shfl_sync(0xffffffffu, dxq, r, LP);
        const f32x2 dd = pk(d, d), dxx = pk(dx, dx);
        const f32x2 h01 = fma2(exp2_2(mul2(dd, A01)), h[r].pair(0), mul2(dxx, Bv[r].pair(0)));
        const f32x2 h23 = fma2(exp2_2(mul2(dd, A23)), h[r].pair(1), mul2(dxx, Bv[r].pair(1)));
        acc[r] = sum2(fma2(Cv[r].pair(1), h23, mul2(Cv[r].pair(0), h01)));
        const f32x2 o[2] = {h01, h23};
        if (slot[r] >= 0)
            store_vec<float, 4>(state + ((int64_t)slot[r] * a.channels + c) * N + 4 * q, Vec<float, 4>::of_pairs(o), nvalid, vecs);
    }
    // the rows' sums over the channel's lanes: lane q ends with row `which`
    int which = 0;
    float s = fold_lanes<R, LP / 2>(acc, q, which);
    // that sum belongs to lane `which` of the channel, which holds the row's x and z; LP / R lanes hold each
    s = __shfl_sync(0xffffffffu, s, (q % R) * (LP / R), LP);
    if (!own) return;
    int live = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) live |= (r == q && slot[r] >= 0);
    s = fmaf(Dq, xq, s);
    if (a.z != nullptr) s *= zq * sigmoid(zq);
    y[(int64_t)(b0 + q) * a.channels + c] = from_f32<T>(live ? s : 0.f);
}

template <typename T, int LP>
int step_lanes(const SelectiveArgs& a, float* state, const int* slots, int nslots, T* y, int* err, cudaStream_t s) {
    constexpr int R = LP < 4 ? LP : 4;
    const bool vecs = a.dstate % 4 == 0 && aligned_to(state, 16) && aligned_to(a.A, 16), vecb = states_of_four(a, sizeof(T));
    const int tiles = ceil_div(a.channels, 256 / LP);
    launch_begin(kKindSelectiveStep, s);
    // several rows a thread where the batch fills the SMs all the same
    if (a.batch / R * tiles >= 152 * 4)
        selective_step_kernel<T, LP, R><<<dim3(tiles, ceil_div(a.batch, R)), 256, 0, s>>>(a, state, slots, nslots, y, err, vecs, vecb);
    else
        selective_step_kernel<T, LP, 1><<<dim3(tiles, a.batch), 256, 0, s>>>(a, state, slots, nslots, y, err, vecs, vecb);
    return launch_end(kKindSelectiveStep, s);
}

template <typename T>
int step_of(const SelectiveArgs& a, float* state, const int* slots, int nslots, void* y, int* err, cudaStream_t s) {
    T* yt = static_cast<T*>(y);
    switch (selective_lanes(a.dstate)) {
        case 2: return step_lanes<T, 2>(a, state, slots, nslots, yt, err, s);
        case 4: return step_lanes<T, 4>(a, state, slots, nslots, yt, err, s);
        case 8: return step_lanes<T, 8>(a, state, slots, nslots, yt, err, s);
        case 16: return step_lanes<T, 16>(a, state, slots, nslots, yt, err, s);
        case 32: return step_lanes<T, 32>(a, state, slots, nslots, yt, err, s);
        default: return SSD_ERR_UNSUPPORTED;
    }
}

}  // namespace

int selective_chunks(const SelectiveArgs& a, int sms) {
    // blocks of one run without a split, and the split that gives each SM about eight warps
    const int lp = selective_lanes(a.dstate), cc = kWarps * 32 / lp;
    const int64_t blocks = (int64_t)a.batch * a.ngroups * ceil_div(a.channels / a.ngroups, cc);
    if (blocks >= sms) return 1;
    const int64_t want = ceil_div64(3 * sms, blocks);
    const int64_t most = a.seqlen / 128 > 0 ? a.seqlen / 128 : 1;
    return (int)(want < most ? want : most);
}

size_t selective_workspace(const SelectiveArgs& a, int chunks) {
    return chunks > 1 ? (size_t)a.batch * chunks * a.channels * (a.dstate + 1) * sizeof(float) : 0;
}

int launch_selective_forward(const SelectiveArgs& a, int chunks, void* y, float* final_state, float* ws, cudaStream_t s) {
    if (a.dtype == SSD_BF16) return forward_of<__nv_bfloat16>(a, chunks, y, final_state, ws, s);
    if (a.dtype == SSD_F16) return forward_of<__half>(a, chunks, y, final_state, ws, s);
    return forward_of<float>(a, chunks, y, final_state, ws, s);
}

int launch_selective_step(const SelectiveArgs& a, float* state, const int* slots, int nslots, void* y, int* err,
                          cudaStream_t s) {
    if (a.dtype == SSD_BF16) return step_of<__nv_bfloat16>(a, state, slots, nslots, y, err, s);
    if (a.dtype == SSD_F16) return step_of<__half>(a, state, slots, nslots, y, err, s);
    return step_of<float>(a, state, slots, nslots, y, err, s);
}

}  // namespace ssd
