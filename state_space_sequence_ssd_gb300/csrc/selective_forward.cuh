// selective_forward.cuh -- the selective scan with one decay per channel and state entry, forward (compiled once per
// element type: k_selective_bf16.cu, k_selective_f16.cu, k_selective_f32.cu).  Per row b, channel c
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
// (Measured with operands in registers: a packed multiply-add 2.13 clocks, two of them with an exponential 5.6.)
//
// Layout: a lane holds eight state entries of four neighbouring channels, LP lanes share a channel.  Shared memory
// returns 128 bytes a clock to the registers, broadcast or not, so what an entry costs in operands decides: with one
// channel and four entries a lane, B, C and dt took 12 bytes an entry, 12 clocks a warp and SM quarter, and the pass
// 354 us at the size above; four by four they take 4 bytes, four by eight 3, and fewer of the pairs (dt, dt) that the
// packed arithmetic wants have to be made.  The 32 chains of the recurrence keep the pipelines full with two warps on
// an SM quarter.  x, dt, z, B and C come to shared memory as they lie in memory, a tile ahead; dt, its softplus and
// dt x are formed once per token and channel.
//
// The sequence is split into chunks where that fills the SMs: the same kernel first computes each chunk's own end state
// from zero, a hop carries the states across the chunks (the decay over a chunk is exp(A sum dt)), and the second run
// starts every chunk from its true state.  selective_plan weighs the first run's cost against the SMs it fills.
#pragma once

#include "selective.cuh"

namespace ssd {
namespace {

// A block's shape: a lane holds CH channels of ST state entries, LP lanes share the channels.
template <typename T, int CH, int ST, int LP>
struct Tile {
    static constexpr int TS = CH == 4 ? 8 : 16;           // tokens of a tile
    static constexpr int NP = ST * LP;                    // state entries, padded
    static constexpr int E = 16 / sizeof(T);              // elements of a 16-byte copy
    static constexpr int COPY = LP * E / CH > 0 ? LP * E / CH : 1;  // tokens that the block's threads copy at once,
    static constexpr int CONV = 4 * LP / CH;              // and convert at once (vectors of four channels)
    static constexpr int channels(int threads) { return CH * threads / LP; }
    // shared memory in bytes: two tiles of x, dt and z and of B and C as they are in memory, then one tile of dt and dt x
    // of B and of C as float32
    static constexpr int raw(int cc) { return TS * (3 * cc + 2 * NP) * (int)sizeof(T); }
    static constexpr int bytes(int cc) { return 2 * raw(cc) + TS * (2 * cc + 2 * NP) * 4; }
};

// A lane's channels, and its entries, from shared memory
template <int CH>
__device__ __forceinline__ void read_channels(const float* p, float (&o)[CH]) {
    if constexpr (CH == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2*>(p);
        o[0] = v.x; o[1] = v.y;
    }
}
template <int PAIRS>
__device__ __forceinline__ void read_entries(const float* p, f32x2 (&o)[PAIRS]) {
#pragma unroll
    for (int i = 0; i < PAIRS / 2; ++i) {
        const float4 v = reinterpret_cast<const float4*>(p)[i];
        o[2 * i] = pk(v.x, v.y);
        o[2 * i + 1] = pk(v.z, v.w);
    }
}

// VEC: every row of x, dt, z, y, B and C is whole 16-byte pieces, copied without a register between.
// PAD: the lanes hold more entries than there are.  Those have A = B = C = 0 and stay zero, until dt x is infinite: zero
// times that is NaN, and so would be y.  A tile with such a value, told by the barrier that it has anyway, goes through a
// loop that sets them to zero again at each token.  (A first run's entries past the last are not stored, so it needs none.)
template <typename T, int CH, int ST, int LP, bool STATE_ONLY, bool VEC, bool PAD>
__global__ void __launch_bounds__(128, 3) selective_kernel(SelectiveArgs a, int chunk, int nchunks, T* __restrict__ y,
                                                           float* __restrict__ final_state, float* hops,
                                                           float* __restrict__ dtsum) {
    using K = Tile<T, CH, ST, LP>;
    constexpr int TS = K::TS, NP = K::NP, E = K::E, PAIRS = ST / 2;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, threads = blockDim.x;
    const int CC = K::channels(threads);  // channels of the block
    const int per = a.channels / a.ngroups, tiles = (per + CC - 1) / CC;
    const int grp = blockIdx.x / tiles, cb = (blockIdx.x % tiles) * CC, g0 = grp * per + cb;
    const int b = blockIdx.z, part = blockIdx.y, N = a.dstate;
    const int len = row_length(a.lengths, b, a.seqlen);
    const int tb = part * chunk, te = min(tb + chunk, a.seqlen), last = min(len, te);
    const int nc = min(CC, per - cb);
    const int64_t n = (int64_t)a.channels * N;
    const bool gated = !STATE_ONLY && a.z != nullptr;

    // the tiles as they are in memory (x, dt, z: TS x CC each; B, C: TS x NP each; twice), and as the loop takes them
    T* raw = reinterpret_cast<T*>(smem);
    const int buffer = K::raw(CC) / (int)sizeof(T);
    float* s_d = reinterpret_cast<float*>(smem + 2 * K::raw(CC));  // dt; then, token by token, the outputs' sums
    float* s_x = s_d + TS * CC;
    float* s_B = s_x + TS * CC;
    float* s_C = s_B + TS * NP;

    const T* xg = static_cast<const T*>(a.x) + b * a.x_batch + g0;
    const T* dg = static_cast<const T*>(a.dt) + b * a.dt_batch + g0;
    const T* zg = gated ? static_cast<const T*>(a.z) + b * a.z_batch + g0 : xg;
    const T* Bg = static_cast<const T*>(a.B) + b * a.B_batch + (int64_t)grp * N;
    const T* Cg = static_cast<const T*>(a.C) + b * a.C_batch + (int64_t)grp * N;
    // copies: this thread's column and first token of x, dt and z, and its first piece of B and C
    const int col = tid % (CC / E) * E, row = tid / (CC / E);
    const bool mine = col < nc;
    const int64_t xs = K::COPY * a.x_token, ds = K::COPY * a.dt_token, zs = K::COPY * a.z_token;
    const T *xc = xg + (int64_t)(tb + row) * a.x_token + col, *dc = dg + (int64_t)(tb + row) * a.dt_token + col;
    const T* zc = gated ? zg + (int64_t)(tb + row) * a.z_token + col : zg;
    auto fetch = [&](int t0, int buf) {
        T* to = raw + buf * buffer;
        if constexpr (VEC) {
            T* at = to + row * CC + col;
            const T *xi = xc, *di = dc, *zi = zc;
#pragma unroll
            for (int i = 0; i < (TS + K::COPY - 1) / K::COPY; ++i) {
                if (TS % K::COPY == 0 || row + i * K::COPY < TS) {
                    const bool live = mine && t0 + row + i * K::COPY < last;
                    copy16(at + i * K::COPY * CC, live ? xi : xg, live);
                    copy16(at + (TS + i * K::COPY) * CC, live ? di : dg, live);
                    if (gated) copy16(at + (2 * TS + i * K::COPY) * CC, live ? zi : zg, live);
                    xi += xs;
                    di += ds;
                    zi += zs;
                }
            }
            xc += TS * a.x_token;
            dc += TS * a.dt_token;
            if (gated) zc += TS * a.z_token;
        } else {
            // rows that are not whole vectors: a column's tokens at a time, their loads in flight together
            for (int c = tid; c < CC; c += threads) {
                T vx[TS], vd[TS], vz[TS];
                const T *xi = xg + (int64_t)t0 * a.x_token + c, *di = dg + (int64_t)t0 * a.dt_token + c;
                const T* zi = gated ? zg + (int64_t)t0 * a.z_token + c : xg;
#pragma unroll
                for (int t = 0; t < TS; ++t) {
                    const bool live = t0 + t < last && c < nc;
                    vx[t] = live ? *xi : from_f32<T>(0.f);
                    vd[t] = live ? *di : from_f32<T>(0.f);
                    vz[t] = live && gated ? *zi : from_f32<T>(0.f);
                    xi += a.x_token;
                    di += a.dt_token;
                    if (gated) zi += a.z_token;
                }
#pragma unroll
                for (int t = 0; t < TS; ++t) {
                    to[t * CC + c] = vx[t];
                    to[(TS + t) * CC + c] = vd[t];
                    to[(2 * TS + t) * CC + c] = vz[t];
                }
            }
        }
        T* bc = to + 3 * TS * CC;
        if constexpr (VEC) {
            constexpr int ROW = NP / E, PART = TS * ROW;  // copies of a token's B, and of all of them
            for (int i = tid; i < (STATE_ONLY ? 1 : 2) * PART; i += threads) {
                const bool isC = i >= PART;
                const int j = isC ? i - PART : i, t = t0 + j / ROW, e = j % ROW * E;
                const bool live = t < last && e < N;
                const T* from = isC ? Cg + (int64_t)t * a.C_token + e : Bg + (int64_t)t * a.B_token + e;
                copy16(bc + i * E, live ? from : Bg, live);
            }
        } else {
            for (int i = tid; i < (STATE_ONLY ? 1 : 2) * TS * NP; i += threads) {
                const bool isC = i >= TS * NP;
                const int j = isC ? i - TS * NP : i, t = t0 + j / NP, e = j % NP;
                const T* from = isC ? Cg + (int64_t)t * a.C_token : Bg + (int64_t)t * a.B_token;
                bc[i] = t < last && e < N ? from[e] : from_f32<T>(0.f);
            }
        }
        copies_commit();
    };
    if (tb < last) fetch(tb, 0);

    // this lane's channels CH qd .. and entries ST q ..
    const int qd = tid / LP, q = tid % LP;
    f32x2 A[CH][PAIRS], h[CH][PAIRS];
    auto read = [&](const float* p, float scale, f32x2 (&o)[CH][PAIRS]) {
        const bool four = N % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < ST / 4; ++i) {
                const int e = ST * q + 4 * i;
                const Vec<float, 4> v = load_vec<float, 4, true>(p + (int64_t)(g0 + CH * qd + c) * N + e,
                                                                 p != nullptr && CH * qd + c < nc ? N - e : 0, four);
                o[c][2 * i] = mul2(v.pair(0), pk(scale, scale));
                o[c][2 * i + 1] = mul2(v.pair(1), pk(scale, scale));
            }
    };
    read(a.A, kLog2e, A);
    const float* from = nullptr;
    if (!STATE_ONLY) grid_dep_wait();  // the hop, where this run follows it
    if (!STATE_ONLY && nchunks > 1) from = hops + ((int64_t)b * nchunks + part) * n;
    else if (!STATE_ONLY && a.init != nullptr) from = a.init + b * n;
    read(from, 1.f, h);

    // this thread's part of the conversions and outputs: channels 4 v0 .., tokens w0, w0 + CONV, ..
    const int v0 = tid % (CC / 4), w0 = tid / (CC / 4), vc = max(0, nc - 4 * v0);
    float bias[4], Dv[4], dsum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        bias[e] = a.dto.bias != nullptr && e < vc ? a.dto.bias[g0 + 4 * v0 + e] : 0.f;
        Dv[e] = a.D != nullptr && e < vc ? a.D[g0 + 4 * v0 + e] : 0.f;
    }
    const int place = w0 * CC + 4 * v0;  // of its first vector in a tile
    constexpr int CONVS = (TS + K::CONV - 1) / K::CONV;
    T* yp = y + ((int64_t)b * a.seqlen + tb + w0) * a.channels + g0 + 4 * v0;

    int buf = 0;
    int t0 = tb;
    for (; t0 < last; t0 += TS, buf ^= 1) {
        copies_wait<0>();
        __syncthreads();  // the tile's copies have landed; the last tile's sums and inputs are read
        if (t0 + TS < last) fetch(t0 + TS, buf ^ 1);
        const T* in = raw + buf * buffer;
        float undefined = 0.f;  // PAD: not zero once a dt x is not finite
        if (w0 < TS) {
            // all of the thread's vectors side by side: each value's dt is a chain of a dozen dependent instructions
            float d[4 * CONVS];
            Vec<T, 4> xv[CONVS];
#pragma unroll
            for (int i = 0; i < CONVS; ++i) {
                const int at = place + i * K::CONV * CC;
                xv[i] = load_vec<T, 4, true>(in + at, 4, true);
                const Vec<T, 4> dt = load_vec<T, 4, true>(in + TS * CC + at, 4, true);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[4 * i + e] = dt.get(e) + bias[e];
            }
            effective<true>(d, a.dto);
#pragma unroll
            for (int i = 0; i < CONVS; ++i) {
                const int at = place + i * K::CONV * CC;
                const bool live = t0 + w0 + i * K::CONV < last;  // dt = 0 keeps the state
                float dx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d[4 * i + e] = live ? d[4 * i + e] : 0.f;
                    dx[e] = d[4 * i + e] * xv[i].get(e);
                    if (STATE_ONLY) dsum[e] += d[4 * i + e];
                    if (PAD) undefined = fmaf(0.f, dx[e], undefined);
                }
                *reinterpret_cast<float4*>(s_d + at) = make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
                *reinterpret_cast<float4*>(s_x + at) = make_float4(dx[0], dx[1], dx[2], dx[3]);
            }
        }
        for (int i = tid; i < (STATE_ONLY ? 1 : 2) * TS * NP / 4; i += threads) {  // s_C follows s_B
            const Vec<T, 4> v = load_vec<T, 4, true>(in + 3 * TS * CC + 4 * i, 4, true);
            reinterpret_cast<float4*>(s_B)[i] = make_float4(v.get(0), v.get(1), v.get(2), v.get(3));
        }
        bool clear = false;
        if (PAD) clear = __syncthreads_or(undefined != 0.f) != 0;
        else __syncthreads();
        const int steps = last - t0 < TS ? last - t0 : TS;  // none for a tile past the length
        float d[CH], x[CH];
        f32x2 B[PAIRS];
        read_channels(s_d + CH * qd, d);
        read_channels(s_x + CH * qd, x);
        read_entries(s_B + ST * q, B);
        auto token = [&](int t, auto clearing) {
            // the next token's operands, before this one's sums are stored over dt
            const int up = t + 1 < TS ? t + 1 : 0;
            float dn[CH], xn[CH];
            f32x2 Bn[PAIRS], C[PAIRS];
            read_channels(s_d + up * CC + CH * qd, dn);
            read_channels(s_x + up * CC + CH * qd, xn);
            read_entries(s_B + up * NP + ST * q, Bn);
            if (!STATE_ONLY) read_entries(s_C + t * NP + ST * q, C);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const f32x2 dd = pk(d[c], d[c]), xx = pk(x[c], x[c]);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) h[c][i] = fma2(exp2_2(mul2(dd, A[c][i])), h[c][i], mul2(xx, B[i]));
                if constexpr (decltype(clearing)::value) {
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        float lo, hi;
                        unpk(h[c][i], lo, hi);
                        h[c][i] = pk(ST * q + 2 * i < N ? lo : 0.f, ST * q + 2 * i + 1 < N ? hi : 0.f);
                    }
                }
            }
            if (!STATE_ONLY) {
                float v[CH];
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    f32x2 s = mul2(C[0], h[c][0]);
#pragma unroll
                    for (int i = 1; i < PAIRS; ++i) s = fma2(C[i], h[c][i], s);
                    v[c] = sum2(s);
                }
                int which = 0;  // over the channels' lanes, each ending with one of the channels (or with several)
                fold_between<CH, LP / 2, 1>(v, q, which);
                // every lane of these channels has read the token's dt: they are lanes of one warp
                if (LP <= CH || (q & ((LP > CH ? LP / CH : 1) - 1)) == 0) {
#pragma unroll
                    for (int e = 0; e < (LP >= CH ? 1 : CH / LP); ++e) s_d[t * CC + CH * qd + which + e] = v[e];
                }
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) { d[c] = dn[c]; x[c] = xn[c]; }
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) B[i] = Bn[i];
        };
        if (PAD && clear) {
#pragma unroll 1
            for (int t = 0; t < steps; ++t) token(t, std::integral_constant<bool, PAD>());
        } else {
#pragma unroll 2
            for (int t = 0; t < steps; ++t) token(t, std::false_type());
        }
        if (!STATE_ONLY) {
            __syncthreads();
            if (w0 < TS) {
                float o[CONVS][4];
#pragma unroll
                for (int i = 0; i < CONVS; ++i) {
                    const int at = place + i * K::CONV * CC;
                    const Vec<T, 4> xv = load_vec<T, 4, true>(in + at, 4, true);
                    const float4 s = *reinterpret_cast<const float4*>(s_d + at);
                    const float sums[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] = fmaf(Dv[e], xv.get(e), sums[e]);
                }
                if (gated) {
#pragma unroll
                    for (int i = 0; i < CONVS; ++i) {
                        const Vec<T, 4> z = load_vec<T, 4, true>(in + 2 * TS * CC + place + i * K::CONV * CC, 4, true);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float zv = z.get(e);
                            o[i][e] *= zv * sigmoid(zv);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < CONVS; ++i) {
                    const int t = t0 + w0 + i * K::CONV;
                    const Vec<T, 4> out = t < last ? Vec<T, 4>::of(o[i]) : Vec<T, 4>::zero();
                    store_vec<T, 4>(yp + (int64_t)(i * K::CONV) * a.channels, out, t < te ? vc : 0, VEC);
                }
            }
            yp += (int64_t)TS * a.channels;
        }
    }
    if (!STATE_ONLY) {  // the tiles past the row's length
        for (int t = t0 + w0; t < te; t += K::CONV) {
            store_vec<T, 4>(yp, Vec<T, 4>::zero(), vc, VEC);
            yp += (int64_t)K::CONV * a.channels;
        }
    }
    float* to = nullptr;
    if (STATE_ONLY) to = hops + ((int64_t)b * nchunks + part + 1) * n;  // carried into the next chunk
    else if (final_state != nullptr && te == a.seqlen) to = final_state + b * n;
    if (to != nullptr) {
        const bool four = N % 4 == 0 && (reinterpret_cast<uintptr_t>(to) & 15) == 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < ST / 4; ++i) {
                const int e = ST * q + 4 * i;
                const f32x2 o[2] = {h[c][2 * i], h[c][2 * i + 1]};
                store_vec<float, 4>(to + (int64_t)(g0 + CH * qd + c) * N + e, Vec<float, 4>::of_pairs(o),
                                    CH * qd + c < nc ? N - e : 0, four);
            }
    }
    if (STATE_ONLY) {
        // sum of dt over the chunk, per channel: over the CONV threads of one vector, in order
        copies_wait<0>();
        __syncthreads();
        if (w0 < TS) *reinterpret_cast<float4*>(s_d + place) = make_float4(dsum[0], dsum[1], dsum[2], dsum[3]);
        __syncthreads();
        for (int c = tid; c < nc; c += threads) {
            float s = 0.f;
            for (int r = 0; r < K::CONV && r < TS; ++r) s += s_d[r * CC + c];
            dtsum[((int64_t)b * nchunks + part) * a.channels + g0 + c] = s;
        }
    }
}

template <typename T, int CH, int ST, int LP>
int forward_shape(const SelectiveArgs& a, const SelectiveShape& f, int chunks, T* y, float* final_state, float* ws, cudaStream_t s) {
    using K = Tile<T, CH, ST, LP>;
    const int tiles = a.ngroups * ceil_div(a.channels / a.ngroups, f.cc);
    const int chunk = ceil_div(ceil_div(a.seqlen, chunks), K::TS) * K::TS;
    const int nchunks = ceil_div(a.seqlen, chunk);
    const int smem = K::bytes(f.cc);
    float* hops = ws;
    float* dtsum = ws == nullptr ? nullptr : ws + (int64_t)a.batch * nchunks * a.channels * a.dstate;
    auto go = [&](auto kernel, int parts, bool follows) {
        int r = ensure_smem_limit(reinterpret_cast<const void*>(kernel), K::bytes(K::channels(128)));
        if (r != SSD_OK) return r;
        launch_begin(kKindSelective, s);
        const dim3 grid(tiles, parts, a.batch);
        if (follows) launch_dependent(kernel, grid, dim3(f.threads), smem, s, a, chunk, nchunks, y, final_state, hops, dtsum);
        else kernel<<<grid, f.threads, smem, s>>>(a, chunk, nchunks, y, final_state, hops, dtsum);
        return launch_end(kKindSelective, s);
    };
    constexpr bool WHOLE = K::NP % K::E == 0;  // the padded entries are whole copies
    const bool vec = WHOLE && rows_of(a, K::E, y, nullptr, sizeof(T)) && f.cc % K::E == 0 && states_of(a, K::E, sizeof(T));
    int r = SSD_OK;
    if (nchunks > 1) {
        if constexpr (WHOLE)
            if (vec) r = go(selective_kernel<T, CH, ST, LP, true, true, false>, nchunks - 1, false);
        if (!vec) r = go(selective_kernel<T, CH, ST, LP, true, false, false>, nchunks - 1, false);
        if (r != SSD_OK) return r;
        r = launch_selective_hop(a, nchunks, hops, dtsum, s);
        if (r != SSD_OK) return r;
    }
    const bool pad = a.dstate < K::NP;
    if constexpr (WHOLE) {
        if (vec) return pad ? go(selective_kernel<T, CH, ST, LP, false, true, true>, nchunks, nchunks > 1)
                            : go(selective_kernel<T, CH, ST, LP, false, true, false>, nchunks, nchunks > 1);
    }
    return pad ? go(selective_kernel<T, CH, ST, LP, false, false, true>, nchunks, nchunks > 1)
               : go(selective_kernel<T, CH, ST, LP, false, false, false>, nchunks, nchunks > 1);
}

template <typename T>
int forward_of(const SelectiveArgs& a, const SelectivePlan& p, void* y, float* final_state, float* ws, cudaStream_t s) {
    T* yt = static_cast<T*>(y);
    const SelectiveShape f = selective_shape(a, p.wide);
    if (!p.wide) {
        switch (f.lp) {
            case 1: return forward_shape<T, 2, 4, 1>(a, f, p.chunks, yt, final_state, ws, s);
            case 2: return forward_shape<T, 2, 4, 2>(a, f, p.chunks, yt, final_state, ws, s);
            case 4: return forward_shape<T, 2, 4, 4>(a, f, p.chunks, yt, final_state, ws, s);
            default: return SSD_ERR_UNSUPPORTED;
        }
    }
    switch (f.lp) {
        case 1: return forward_shape<T, 4, 8, 1>(a, f, p.chunks, yt, final_state, ws, s);
        case 2: return forward_shape<T, 4, 8, 2>(a, f, p.chunks, yt, final_state, ws, s);
        case 4: return forward_shape<T, 4, 8, 4>(a, f, p.chunks, yt, final_state, ws, s);
        case 8: return forward_shape<T, 4, 8, 8>(a, f, p.chunks, yt, final_state, ws, s);
        case 16: return forward_shape<T, 4, 8, 16>(a, f, p.chunks, yt, final_state, ws, s);
        default: return SSD_ERR_UNSUPPORTED;
    }
}

}  // namespace
}  // namespace ssd
