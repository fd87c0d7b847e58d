// group_norm.cuh -- the norm over groups of a token's channels with its activation, and its gradient; compiled once per element
// type by k_group_norm_{bf16,f16,f32}.cu.
//
//   q    = x silu(z)  where the gate comes first, else x
//   xhat = (q - mean) rstd (the mean left out where rms),   n = xhat weight + bias
//   y    = n, silu(n), or n silu(z) where the gate comes last
//   backward, with g the gradient of n (dy, through the activation), gw = g weight:
//   dq = rstd (gw - mean(gw) - xhat mean(gw xhat)),  dweight = sum g xhat,  dbias = sum g
//   dx = dq (through silu(z) where it comes first), dz = dy n silu'(z) or dq x silu'(z)
//
// A unit is one group of one row.  `lanes` threads (a power of two, at most a block's) share it and hold it in registers, so that
// everything is read once: up to 32 lanes, as for a group per head, the sums take shuffles alone.  Bound by HBM.
#pragma once

#include "norm.cuh"

namespace ssd {
namespace {

// sigmoid of two values.  Packed where it can be: its two constants stay in registers over a thread's many values.
__device__ __forceinline__ f32x2 sigmoid_pair(f32x2 v) {
    float a, b;
    unpk(add2(exp2_2(mul2(v, pk(-kLog2e, -kLog2e))), pk(1.f, 1.f)), a, b);
    return pk(rcp_fast(a), rcp_fast(b));
}
// silu(v) = v sigmoid(v) and its slope
__device__ __forceinline__ f32x2 slope_of(f32x2 v, f32x2 sig) {
    const f32x2 one = pk(1.f, 1.f);
    return mul2(sig, fma2(v, fma2(sig, pk(-1.f, -1.f), one), one));
}

__device__ __forceinline__ float unpk_low(f32x2 v) {
    float a, b;
    unpk(v, a, b);
    return a;
}

// Row and group of unit u (units that fit 32 bits, as all but the longest do, are divided there).
__device__ __forceinline__ void unit_of(int64_t u, int groups, int64_t& row, int& group) {
    if (u <= 0xffffffffll) {
        row = (uint32_t)u / (uint32_t)groups;
        group = (int)((uint32_t)u - (uint32_t)row * (uint32_t)groups);
    } else {
        row = u / groups;
        group = (int)(u - row * groups);
    }
}

// Rows and groups that are whole 16-byte vectors are read in those (V = 8 or 4); others in pairs, an element at a time.
template <int V>
constexpr bool kWhole = V > 2;
// EVEN, for the others: groups are whole pairs, and outputs and weights aligned to pairs.
template <typename T, int V, bool EVEN>
__device__ __forceinline__ Vec<T, V> load_part(const T* p, int valid) {
    if constexpr (!kWhole<V> && EVEN) {
        Vec<T, V> r = Vec<T, V>::zero();
        if (valid > 0) {
            r.w[0] = bits_at(p);
            if constexpr (sizeof(T) == 4) r.w[1] = bits_at(p + 1);
            else r.w[0] |= bits_at(p + 1) << 16;
        }
        return r;
    } else {
        return load_vec<T, V>(p, valid, kWhole<V>);
    }
}
template <int V, bool EVEN>
__device__ __forceinline__ void load_weights(const float* p, int c, int per, bool vecw, float otherwise, f32x2 (&o)[(V + 1) / 2]) {
    if constexpr (!kWhole<V> && EVEN) {
        float2 q = make_float2(otherwise, otherwise);
        if (p != nullptr && c < per) q = __ldg(reinterpret_cast<const float2*>(p + c));
        o[0] = pk(q.x, q.y);
    } else {
        load_columns<V>(p, c, per, vecw, otherwise, o);
    }
}

// Thread `lane` of a unit holds columns (lane + lanes i) V .. of its group.
// Eight pairs a thread take 64 registers where they are held to that, up to 80 where not (20000 x 330 of bfloat16 in 3 groups, gated behind:
// 14.4 us, 15.6 with 80).
template <typename T, int V, int NV, int GATE, bool EVEN>
__global__ void __launch_bounds__(kThreads, !kWhole<V> && NV == 8 ? 4 : 0) group_forward_kernel(GroupNormArgs g, int lanes, T* __restrict__ y, float* __restrict__ mean,
                                                                 float* __restrict__ rstd, bool vecw) {
    constexpr int P = (V + 1) / 2;
    __shared__ float2 buf[2][kThreads / 32];
    const int lane = threadIdx.x & (lanes - 1), per = g.width / g.groups;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    const bool live = unit < g.rows * g.groups;
    int64_t row = 0;
    int group = 0;
    if (live) unit_of(unit, g.groups, row, group);
    const int base = group * per;
    const T* x = static_cast<const T*>(g.x) + row * g.x_row + base;
    const T* z = static_cast<const T*>(g.z) + (GATE >= kGateAfter ? row * g.z_row + base : 0);
    Vec<T, V> rx[NV], rz[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + lanes * i) * V;
        rx[i] = load_part<T, V, EVEN>(x + c, live ? per - c : 0);
        if (GATE >= kGateAfter) rz[i] = load_part<T, V, EVEN>(z + c, live ? per - c : 0);
    }
    f32x2 q[NV][P], s2 = 0ull, v2 = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) {
            q[i][e] = rx[i].pair(e);
            if (GATE == kGateBefore) {
                const f32x2 zz = rz[i].pair(e);
                q[i][e] = mul2(q[i][e], mul2(zz, sigmoid_pair(zz)));
            }
            s2 = add2(s2, q[i][e]);
        }
    const float inv = 1.f / (float)per;
    const float m = g.rms ? 0.f : mean_of(row_sum(sum2(s2), lanes, buf[0]), per, inv);
    const f32x2 m2 = pk(-m, -m);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((lane + lanes * i) * V < per) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                q[i][e] = add2(q[i][e], m2);
                if (!kWhole<V> && !EVEN && (lane + lanes * i) * V + 1 >= per) q[i][e] = pk(unpk_low(q[i][e]), 0.f);  // half a pair
                v2 = fma2(q[i][e], q[i][e], v2);
            }
        }
    const float rs = rsqrtf(fmaf(row_sum(sum2(v2), lanes, buf[1]), inv, g.eps));
    if (!live) return;
    if (lane == 0) {
        if (mean != nullptr) mean[unit] = m;
        if (rstd != nullptr) rstd[unit] = rs;
    }
    T* o = y + row * g.width + base;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + lanes * i) * V;
        if (c >= per) break;
        f32x2 w[P], b[P], out[P];
        load_weights<V, EVEN>(g.weight == nullptr ? nullptr : g.weight + base, c, per, vecw, 1.f, w);
        load_weights<V, EVEN>(g.bias == nullptr ? nullptr : g.bias + base, c, per, vecw, 0.f, b);
#pragma unroll
        for (int e = 0; e < P; ++e) {
            out[e] = fma2(mul2(q[i][e], pk(rs, rs)), w[e], b[e]);
            if (GATE == kGateSilu) out[e] = mul2(out[e], sigmoid_pair(out[e]));
            if (GATE == kGateAfter) {
                const f32x2 zz = rz[i].pair(e);
                out[e] = mul2(out[e], mul2(zz, sigmoid_pair(zz)));
            }
        }
        store_vec<T, V>(o + c, Vec<T, V>::of_pairs(out), per - c, kWhole<V> || EVEN);
    }
}

// The same for many rows of whole vectors: a resident grid whose blocks walk the rows.  A thread keeps its columns, and with them their
// weights; a block holds `side` groups of a row next to one another and kThreads / lanes / side rows at once.  A thread's
// pieces of the next rows are copied to shared memory that it alone reads.  8192 x 4096 of bfloat16 in 8 groups, gated in front:
// 35.0 us (5.8 TB/s; floor 29.7).  On one set of inputs, part of it in L2, 33.7; 41.0 with the kernel above, whose threads spend half their
// instructions on addresses and weights; copies three rows ahead 36.2, four blocks an SM 36.4.
constexpr int kForwardAhead = 2;
constexpr int kWalkers = 3;  // blocks of an SM
template <typename T, int V, int NV, int GATE>
__global__ void __launch_bounds__(kThreads, kWalkers) group_walk_kernel(GroupNormArgs g, int lanes, int side, T* __restrict__ y, float* __restrict__ mean,
                                                                 float* __restrict__ rstd, bool vecw) {
    constexpr int P = V / 2, TENSORS = GATE >= kGateAfter ? 2 : 1;
    constexpr bool Z = GATE >= kGateAfter;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float2 buf[2][kThreads / 32];
    const int lane = threadIdx.x & (lanes - 1), sub = threadIdx.x / lanes, high = kThreads / lanes / side;
    const int per = g.width / g.groups, group = blockIdx.x * side + sub % side, base = group * per;
    const bool here = group < g.groups;
    const float inv = 1.f / (float)per;
    f32x2 w[NV][P], b[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + lanes * i) * V;
        load_columns<V>(g.weight == nullptr ? nullptr : g.weight + (here ? base : 0), c, per, vecw, 1.f, w[i]);
        load_columns<V>(g.bias == nullptr ? nullptr : g.bias + (here ? base : 0), c, per, vecw, 0.f, b[i]);
    }
    uint4* ring = reinterpret_cast<uint4*>(smem) + threadIdx.x;
    const T *x = static_cast<const T*>(g.x) + (here ? base : 0), *z = Z ? static_cast<const T*>(g.z) + (here ? base : 0) : nullptr;
    auto fetch = [&](int64_t row, int turn) {
        const bool live = here && row < g.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + lanes * i) * V;
            const bool in = live && c < per;
            uint4* to = ring + (turn * NV + i) * TENSORS * kThreads;
            copy16(to, in ? x + row * g.x_row + c : x, in);
            if (Z) copy16(to + kThreads, in ? z + row * g.z_row + c : z, in);
        }
        copies_commit();
    };
    const int64_t step = (int64_t)gridDim.y * high;
    int64_t row = (int64_t)blockIdx.y * high + sub / side;
#pragma unroll
    for (int k = 0; k < kForwardAhead; ++k) fetch(row + k * step, k);
    int turn = 0, flip = 0;  // sums that follow one another take turns in buf, with a mean or without
    for (int64_t r0 = (int64_t)blockIdx.y * high; r0 < g.rows; r0 += step, row += step) {
        Vec<T, V> cz[NV];
        f32x2 q[NV][P], s2 = 0ull, v2 = 0ull;
        copies_wait<kForwardAhead - 1>();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint4* from = ring + (turn * NV + i) * TENSORS * kThreads;
            Vec<T, V> cx;
            const uint4 u = from[0];
            cx.w[0] = u.x; cx.w[1] = u.y; cx.w[2] = u.z; cx.w[3] = u.w;
            if (Z) {
                const uint4 u2 = from[kThreads];
                cz[i].w[0] = u2.x; cz[i].w[1] = u2.y; cz[i].w[2] = u2.z; cz[i].w[3] = u2.w;
            }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                q[i][e] = cx.pair(e);
                if (GATE == kGateBefore) {
                    const f32x2 zz = cz[i].pair(e);
                    q[i][e] = mul2(q[i][e], mul2(zz, sigmoid_pair(zz)));
                }
            }
        }
        fetch(row + kForwardAhead * step, turn);
        if (++turn == kForwardAhead) turn = 0;
        float m = 0.f;
        if (!g.rms) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < P; ++e) s2 = add2(s2, q[i][e]);
            m = mean_of(row_sum(sum2(s2), lanes, buf[flip ^= 1]), per, inv);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < P; ++e) q[i][e] = add2(q[i][e], pk(-m, -m));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((lane + lanes * i) * V < per) {
#pragma unroll
                for (int e = 0; e < P; ++e) v2 = fma2(q[i][e], q[i][e], v2);
            }
        const float rs = rsqrtf(fmaf(row_sum(sum2(v2), lanes, buf[flip ^= 1]), inv, g.eps));
        if (!here || row >= g.rows) continue;
        if (lane == 0) {
            if (mean != nullptr) mean[row * g.groups + group] = m;
            if (rstd != nullptr) rstd[row * g.groups + group] = rs;
        }
        T* o = y + row * g.width + base;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + lanes * i) * V;
            if (c >= per) break;
            f32x2 out[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                out[e] = fma2(mul2(q[i][e], pk(rs, rs)), w[i][e], b[i][e]);
                if (GATE == kGateSilu) out[e] = mul2(out[e], sigmoid_pair(out[e]));
                if (GATE == kGateAfter) {
                    const f32x2 zz = cz[i].pair(e);
                    out[e] = mul2(out[e], mul2(zz, sigmoid_pair(zz)));
                }
            }
            store_vec<T, V>(o + c, Vec<T, V>::of_pairs(out), per - c, true);
        }
    }
    copies_wait<0>();
}

// One value of q from memory.
template <typename T>
__device__ __forceinline__ float gated_value(const GroupNormArgs& g, int64_t row, int c) {
    const float x = to_f32<T>(static_cast<const T*>(g.x)[row * g.x_row + c]);
    if (g.gate != kGateBefore) return x;
    const float z = to_f32<T>(static_cast<const T*>(g.z)[row * g.z_row + c]);
    return x * (z * sigmoid(z));
}

// Groups that do not fit the registers, a block each: read again (from L2) for each sum and the output.
template <typename T>
__global__ void __launch_bounds__(kThreads) group_forward_wide_kernel(GroupNormArgs g, T* __restrict__ y, float* __restrict__ mean,
                                                                      float* __restrict__ rstd) {
    __shared__ float2 buf[2][kThreads / 32];
    const int per = g.width / g.groups;
    int64_t row;
    int group;
    unit_of(blockIdx.x, g.groups, row, group);
    const int base = group * per;
    const float inv = 1.f / (float)per;
    float s = 0.f, q = 0.f;
    if (!g.rms) {
#pragma unroll 4
        for (int c = threadIdx.x; c < per; c += kThreads) s += gated_value<T>(g, row, base + c);
    }
    const float m = g.rms ? 0.f : mean_of(row_sum(s, kThreads, buf[0]), per, inv);
#pragma unroll 4
    for (int c = threadIdx.x; c < per; c += kThreads) {
        const float d = gated_value<T>(g, row, base + c) - m;
        q = fmaf(d, d, q);
    }
    const float rs = rsqrtf(fmaf(row_sum(q, kThreads, buf[1]), inv, g.eps));
    if (threadIdx.x == 0) {
        if (mean != nullptr) mean[blockIdx.x] = m;
        if (rstd != nullptr) rstd[blockIdx.x] = rs;
    }
#pragma unroll 4
    for (int c = threadIdx.x; c < per; c += kThreads) {
        float n = fmaf((gated_value<T>(g, row, base + c) - m) * rs, g.weight != nullptr ? g.weight[base + c] : 1.f, g.bias != nullptr ? g.bias[base + c] : 0.f);
        if (g.gate == kGateSilu) n *= sigmoid(n);
        if (g.gate == kGateAfter) {
            const float z = to_f32<T>(static_cast<const T*>(g.z)[row * g.z_row + base + c]);
            n *= z * sigmoid(z);
        }
        y[row * g.width + base + c] = from_f32<T>(n);
    }
}

// A block holds `side` groups of a row next to one another and kThreads / lanes / side rows at once, and walks the rows a grid's
// height apart; its columns' sums stay in registers.  Whole vectors of the next rows are copied to shared memory that their thread
// alone reads, so that they need neither registers nor barriers on their way.  8192 x 4096 of bfloat16 in 8 groups, gated in front, with
// the sums of the blocks 59 us (5.7 TB/s; floor 49.5); values held between the two passes over a row instead of computed twice
// 74, three rows ahead 68, three blocks an SM 68.
constexpr int kRowsAhead = 2;
template <typename T, int V, int NV, int GATE, bool BIAS, bool EVEN>
__global__ void __launch_bounds__(kThreads, 2) group_backward_kernel(GroupNormArgs g, int lanes, int side, const float* __restrict__ mean,
                                                                     const float* __restrict__ rstd, const T* __restrict__ dy, int64_t dy_row,
                                                                     T* __restrict__ dx, T* __restrict__ dz, float* __restrict__ partial, bool vecw) {
    constexpr int P = (V + 1) / 2, TENSORS = GATE >= kGateAfter ? 3 : 2;
    constexpr bool Z = GATE >= kGateAfter, PRE = GATE == kGateSilu || GATE == kGateAfter;
    extern __shared__ __align__(16) unsigned char smem[];  // copies; at the end rows at once x 2 x the block's columns
    __shared__ float2 buf[2][kThreads / 32];
    const int lane = threadIdx.x & (lanes - 1), sub = threadIdx.x / lanes, high = kThreads / lanes / side;
    const int per = g.width / g.groups, group = blockIdx.x * side + sub % side, base = group * per;
    const bool here = group < g.groups;
    const float inv = 1.f / (float)per;
    f32x2 w[NV][P], b[PRE && BIAS ? NV : 1][P], dw[NV][P], db[BIAS ? NV : 1][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + lanes * i) * V;
        load_weights<V, EVEN>(g.weight == nullptr ? nullptr : g.weight + (here ? base : 0), c, per, vecw, 1.f, w[i]);
        if (PRE && BIAS) load_weights<V, EVEN>(g.bias == nullptr ? nullptr : g.bias + (here ? base : 0), c, per, vecw, 0.f, b[i]);
#pragma unroll
        for (int e = 0; e < P; ++e) dw[i][e] = db[BIAS ? i : 0][e] = 0ull;
    }
    const T *x = static_cast<const T*>(g.x), *z = static_cast<const T*>(g.z);
    uint4* ring = reinterpret_cast<uint4*>(smem) + threadIdx.x;
    float* stats = reinterpret_cast<float*>(smem + (kWhole<V> ? kRowsAhead * NV * TENSORS * kThreads * 16 : 0)) + threadIdx.x;
    auto fetch = [&](int64_t row, int turn) {
        const bool live = here && row < g.rows;
        if (kWhole<V>) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + lanes * i) * V;
                const bool in = live && c < per;
                uint4* to = ring + (turn * NV + i) * TENSORS * kThreads;
                copy16(to, in ? x + row * g.x_row + base + c : x, in);
                copy16(to + kThreads, in ? dy + row * dy_row + base + c : dy, in);
                if (Z) copy16(to + 2 * kThreads, in ? z + row * g.z_row + base + c : z, in);
            }
        }
        if (live) {
            copy4(stats + turn * 2 * kThreads, rstd + row * g.groups + group);
            if (mean != nullptr) copy4(stats + (turn * 2 + 1) * kThreads, mean + row * g.groups + group);
        }
        copies_commit();
    };
    struct Part {
        Vec<T, V> x, dy, z;
    };
    const int64_t step = (int64_t)gridDim.y * high;
    int64_t row = (int64_t)blockIdx.y * high + sub / side;
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k) fetch(row + k * step, k);
    int turn = 0, flip = 0;
    for (int64_t r0 = (int64_t)blockIdx.y * high; r0 < g.rows; r0 += step, row += step, turn = turn + 1 == kRowsAhead ? 0 : turn + 1) {
        copies_wait<kRowsAhead - 1>();
        const bool current = here && row < g.rows;
        const float rs = current ? stats[turn * 2 * kThreads] : 0.f, mn = current && mean != nullptr ? stats[(turn * 2 + 1) * kThreads] : 0.f;
        const f32x2 rs2 = pk(rs, rs);
        // Both passes over the row take it from shared memory (pairs: from L1) and compute the same from it: what the sums stand
        // between would not fit the registers.
        auto part = [&](int i) {
            Part p;
            if constexpr (kWhole<V>) {
                const uint4* from = ring + (turn * NV + i) * TENSORS * kThreads;
                auto take = [&](Vec<T, V>& v, const uint4& u) {
                    v.w[0] = u.x;
                    v.w[1] = u.y;
                    v.w[2] = u.z;
                    v.w[3] = u.w;
                };
                take(p.x, from[0]);
                take(p.dy, from[kThreads]);
                if (Z) take(p.z, from[2 * kThreads]);
            } else {
                const int64_t at = current ? row : 0, off = current ? base : 0;
                const int c = (lane + lanes * i) * V, left = current ? per - c : 0;
                p.x = load_part<T, V, EVEN>(x + at * g.x_row + off + c, left);
                p.dy = load_part<T, V, EVEN>(dy + at * dy_row + off + c, left);
                if (Z) p.z = load_part<T, V, EVEN>(z + at * g.z_row + off + c, left);
            }
            return p;
        };
        struct Value {
            f32x2 xhat, g, n, silu, sig;  // n with an activation behind the norm; the last two of the gate
        };
        auto value = [&](const Part& p, int i, int e) {
            Value v;
            if constexpr (Z) {
                const f32x2 zz = p.z.pair(e);
                v.sig = sigmoid_pair(zz);
                v.silu = mul2(zz, v.sig);
            }
            // The difference first: q rstd - (mean rstd) would shift the whole group by that product's rounding.
            if constexpr (GATE == kGateBefore) v.xhat = mul2(add2(mul2(p.x.pair(e), v.silu), pk(-mn, -mn)), rs2);
            else v.xhat = mul2(pair_plus(p.x, e, -mn), rs2);
            v.g = p.dy.pair(e);  // zero past the group's end
            if constexpr (PRE) v.n = BIAS ? fma2(v.xhat, w[i][e], b[BIAS ? i : 0][e]) : mul2(v.xhat, w[i][e]);
            if constexpr (GATE == kGateSilu) v.g = mul2(v.g, slope_of(v.n, sigmoid_pair(v.n)));
            if constexpr (GATE == kGateAfter) v.g = mul2(v.g, v.silu);
            return v;
        };
        f32x2 s1 = 0ull, s2 = 0ull;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Part p = part(i);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const Value v = value(p, i, e);
                const f32x2 gw = mul2(v.g, w[i][e]);
                if (BIAS) db[BIAS ? i : 0][e] = add2(db[BIAS ? i : 0][e], v.g);
                dw[i][e] = fma2(v.g, v.xhat, dw[i][e]);
                s1 = add2(s1, gw);
                s2 = fma2(gw, v.xhat, s2);
            }
        }
        const float2 s = row_sums(make_float2(sum2(s1), sum2(s2)), lanes, buf[flip ^= 1]);
        asm volatile("" ::: "memory");  // the second pass reads again
        if (current) {
            const float k1 = g.rms ? 0.f : -s.x * inv * rs, k2 = -s.y * inv * rs;
            T *ox = dx + row * g.width + base, *oz = Z ? dz + row * g.width + base : nullptr;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + lanes * i) * V;
                if (c >= per) break;
                const Part p = part(i);
                f32x2 o1[P], o2[P];
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const Value v = value(p, i, e);
                    o1[e] = fma2(mul2(v.g, w[i][e]), rs2, fma2(v.xhat, pk(k2, k2), pk(k1, k1)));
                    if constexpr (GATE == kGateBefore) {
                        o2[e] = mul2(mul2(o1[e], p.x.pair(e)), slope_of(p.z.pair(e), v.sig));
                        o1[e] = mul2(o1[e], v.silu);
                    }
                    if constexpr (GATE == kGateAfter) o2[e] = mul2(mul2(p.dy.pair(e), v.n), slope_of(p.z.pair(e), v.sig));
                }
                store_vec<T, V>(ox + c, Vec<T, V>::of_pairs(o1), per - c, kWhole<V> || EVEN);
                if constexpr (Z) store_vec<T, V>(oz + c, Vec<T, V>::of_pairs(o2), per - c, kWhole<V> || EVEN);
            }
        }
        fetch(row + kRowsAhead * step, turn);
    }
    copies_wait<0>();
    if (partial == nullptr) return;
    // the block's columns, one sum for all rows at once
    __syncthreads();  // the copies' place is the sums' now
    float* sums = reinterpret_cast<float*>(smem);
    const int columns = side * per, first = blockIdx.x * columns;
    float* out = partial + (int64_t)blockIdx.y * 2 * g.width;
    float* to = sums + (sub / side) * 2 * columns + (sub % side) * per;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = (lane + lanes * i) * V + e;
            float p, q;
            unpk(dw[i][e / 2], p, q);
            const float a = e & 1 ? q : p;
            unpk(db[BIAS ? i : 0][e / 2], p, q);
            const float d = e & 1 ? q : p;
            if (c >= per || !here) continue;
            if (high == 1) {
                out[base + c] = a;
                if (BIAS) out[g.width + base + c] = d;
            } else {
                to[c] = a;
                to[columns + c] = d;
            }
        }
    if (high == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < columns; c += kThreads) {
        if (first + c >= g.width) continue;
        float p = 0.f, q = 0.f;
        for (int k = 0; k < high; ++k) {
            p += sums[k * 2 * columns + c];
            q += sums[k * 2 * columns + columns + c];
        }
        out[first + c] = p;
        if (BIAS) out[g.width + first + c] = q;
    }
}

// Groups wider than the registers hold: a block per row and group at a time, x, z and dy read twice (the second time from L2), the
// columns' sums kept in the block's row of `partial`.
template <typename T>
__global__ void __launch_bounds__(kThreads) group_backward_wide_kernel(GroupNormArgs g, const float* __restrict__ mean, const float* __restrict__ rstd,
                                                                       const T* __restrict__ dy, int64_t dy_row, T* __restrict__ dx,
                                                                       T* __restrict__ dz, float* __restrict__ partial) {
    __shared__ float2 buf[2][kThreads / 32];
    const int per = g.width / g.groups, base = blockIdx.x * per;
    const float inv = 1.f / (float)per;
    int turn = 0;
    float* sum = partial == nullptr ? nullptr : partial + (int64_t)blockIdx.y * 2 * g.width;
    for (int64_t row = blockIdx.y; row < g.rows; row += gridDim.y) {
        const float m = mean != nullptr ? mean[row * g.groups + blockIdx.x] : 0.f, rs = rstd[row * g.groups + blockIdx.x];
        float n, z, sig;
        auto parts = [&](int c, float& xh, float& gy) {
            xh = (gated_value<T>(g, row, c) - m) * rs;
            gy = to_f32<T>(dy[row * dy_row + c]);
            n = fmaf(xh, g.weight != nullptr ? g.weight[c] : 1.f, g.bias != nullptr ? g.bias[c] : 0.f);
            if (g.gate == kGateSilu) {
                const float s = sigmoid(n);
                gy *= s * fmaf(n, 1.f - s, 1.f);
            }
            if (g.gate >= kGateAfter) {
                z = to_f32<T>(static_cast<const T*>(g.z)[row * g.z_row + c]);
                sig = sigmoid(z);
            }
            if (g.gate == kGateAfter) gy *= z * sig;
        };
        float2 s = make_float2(0.f, 0.f);
        for (int c = base + threadIdx.x; c < base + per; c += kThreads) {
            float xh, gy;
            parts(c, xh, gy);
            const float gw = gy * (g.weight != nullptr ? g.weight[c] : 1.f);
            if (sum != nullptr) {
                const bool first = row == blockIdx.y;
                sum[c] = first ? gy * xh : fmaf(gy, xh, sum[c]);
                sum[g.width + c] = first ? gy : sum[g.width + c] + gy;
            }
            s.x += gw;
            s.y = fmaf(gw, xh, s.y);
        }
        s = row_sums(s, kThreads, buf[turn]);
        turn ^= 1;
        const float s1 = g.rms ? 0.f : s.x * inv, s2 = s.y * inv;
        for (int c = base + threadIdx.x; c < base + per; c += kThreads) {
            float xh, gy;
            parts(c, xh, gy);
            const float gw = gy * (g.weight != nullptr ? g.weight[c] : 1.f);
            float dq = rs * (gw - s1 - xh * s2);
            const int64_t at = row * g.width + c;
            if (g.gate >= kGateAfter) {
                const float slope = sig * fmaf(z, 1.f - sig, 1.f);
                const float other = g.gate == kGateAfter ? to_f32<T>(dy[row * dy_row + c]) * n : dq * to_f32<T>(static_cast<const T*>(g.x)[row * g.x_row + c]);
                dz[at] = from_f32<T>(other * slope);
                if (g.gate == kGateBefore) dq *= z * sig;
            }
            dx[at] = from_f32<T>(dq);
        }
    }
}

// ------------------------------------------------------------------ launches

// Whether rows and groups are whole 16-byte vectors.
template <typename T>
bool in_vectors(const GroupNormArgs& g) {
    constexpr int V = 16 / sizeof(T);
    return g.width / g.groups % V == 0 && g.x_row % V == 0 && (g.z == nullptr || g.z_row % V == 0) && aligned_to(g.x, 16) && aligned_to(g.z, 16);
}

template <typename T, int V, int GATE>
int group_forward_of(const GroupNormArgs& g, void* y, float* mean, float* rstd, cudaStream_t s) {
    constexpr int M = kWhole<V> ? 1 : 4;
    const int64_t units = g.rows * g.groups;
    const int vecs = ceil_div(g.width / g.groups, V), lanes = row_lanes(units, vecs, 2 * M, 1), nv = ceil_div(vecs, lanes);
    const int64_t blocks = ceil_div64(units, kThreads / lanes);
    const bool vecw = aligned_to(g.weight, 16) && aligned_to(g.bias, 16);
    if (blocks > 2147483647) return SSD_ERR_UNSUPPORTED;
    if constexpr (kWhole<V>) {
        // The walk pays from two rows a block (gated in front, bfloat16, one row a thread's group and walk: 608 x 4096 in 8 groups 4.6 and
        // 5.3 us, 1216 7.1 and 6.9, 2432 12.1 and 10.2; in one group 912 x 4096 6.7 and 6.5; 8192 x 4096 in 8 41.0 and 33.7).
        int side = 1;
        while (side < kThreads / lanes && side < g.groups) side *= 2;
        const int slabs = ceil_div(g.groups, side);
        const int64_t high = kThreads / lanes / side, most = ceil_div64(g.rows, high), parts = kWalkers * kSms / slabs;
        if (nv <= 2 && parts > 0 && most >= 2 * parts) {
            int r = SSD_OK;
            launch_begin(kKindGroupNorm, s);
            auto walk = [&](auto kernel, int held) {
                const int smem = kForwardAhead * held * (GATE >= kGateAfter ? 2 : 1) * kThreads * 16;
                if (smem > 32 * 1024) r = ensure_smem_limit(reinterpret_cast<const void*>(kernel), 100 * 1024);  // beside static memory
                if (r == SSD_OK) kernel<<<dim3(slabs, (unsigned)parts), kThreads, smem, s>>>(g, lanes, side, static_cast<T*>(y), mean, rstd, vecw);
            };
            if (nv == 1) walk(group_walk_kernel<T, V, 1, GATE>, 1);
            else walk(group_walk_kernel<T, V, 2, GATE>, 2);
            const int e = launch_end(kKindGroupNorm, s);
            return r != SSD_OK ? r : e;
        }
    }
    launch_begin(kKindGroupNorm, s);
    auto go = [&](auto kernel) { kernel<<<(unsigned)blocks, kThreads, 0, s>>>(g, lanes, static_cast<T*>(y), mean, rstd, vecw); };
    auto held = [&](auto even) {
        constexpr bool EVEN = decltype(even)::value;
        if (nv <= 1 * M) go(group_forward_kernel<T, V, 1 * M, GATE, EVEN>);
        else if (nv <= 2 * M) go(group_forward_kernel<T, V, 2 * M, GATE, EVEN>);
        else go(group_forward_kernel<T, V, 4 * M, GATE, EVEN>);
    };
    const bool even = !kWhole<V> && g.width / g.groups % 2 == 0 && aligned_to(g.weight, 8) && aligned_to(g.bias, 8) && aligned_to(y, 2 * sizeof(T));
    if (nv <= 4 * M && even) held(std::integral_constant<bool, !kWhole<V>>());
    else if (nv <= 4 * M) held(std::false_type());
    else group_forward_wide_kernel<T><<<(unsigned)blocks, kThreads, 0, s>>>(g, static_cast<T*>(y), mean, rstd);
    return launch_end(kKindGroupNorm, s);
}

template <typename T, int V, int GATE>
int group_backward_of(const GroupNormArgs& g, const GroupNormGrads& d, float* partial, int* parts, cudaStream_t s) {
    constexpr int M = kWhole<V> ? 1 : 4;
    const int vecs = ceil_div(g.width / g.groups, V), lanes = row_lanes(g.rows * g.groups, vecs, 2 * M, 1), nv = ceil_div(vecs, lanes);
    const int room = kThreads / lanes;
    int side = 1;
    while (side < room && side < g.groups) side *= 2;
    // Blocks that walk the rows: two an SM over all slabs, none without a row.
    const int high = nv <= 2 * M ? room / side : 1, slabs = nv <= 2 * M ? ceil_div(g.groups, side) : g.groups;
    const int64_t most = ceil_div64(g.rows, high);
    const int want = ceil_div(2 * kSms, slabs), walkers = most < want ? (int)most : want;
    *parts = walkers < *parts ? walkers : *parts;
    const int sums = high == 1 || partial == nullptr ? 0 : high * 2 * side * (g.width / g.groups) * 4;
    const bool vecw = aligned_to(g.weight, 16) && aligned_to(g.bias, 16);
    const T* dy = static_cast<const T*>(d.dy);
    T *dx = static_cast<T*>(d.dx), *dz = static_cast<T*>(d.dz);
    launch_begin(kKindGroupNormBwd, s);
    int r = SSD_OK;
    auto go = [&](auto kernel, int held) {
        const int copies = kRowsAhead * kThreads * ((kWhole<V> ? held * (GATE >= kGateAfter ? 3 : 2) * 16 : 0) + 8), smem = copies > sums ? copies : sums;
        if (smem > 32 * 1024) r = ensure_smem_limit(reinterpret_cast<const void*>(kernel), 100 * 1024);  // beside static memory
        if (r == SSD_OK)
            kernel<<<dim3(slabs, *parts), kThreads, smem, s>>>(g, lanes, side, d.mean, d.rstd, dy, d.dy_row, dx, dz, partial, vecw);
    };
    const bool bias = g.bias != nullptr || d.want_dbias;
    auto held = [&](auto even) {
        constexpr bool EVEN = decltype(even)::value;
        if (nv <= 1 * M) bias ? go(group_backward_kernel<T, V, 1 * M, GATE, true, EVEN>, 1) : go(group_backward_kernel<T, V, 1 * M, GATE, false, EVEN>, 1);
        else bias ? go(group_backward_kernel<T, V, 2 * M, GATE, true, EVEN>, 2) : go(group_backward_kernel<T, V, 2 * M, GATE, false, EVEN>, 2);
    };
    const bool even = !kWhole<V> && g.width / g.groups % 2 == 0 && aligned_to(g.weight, 8) && aligned_to(g.bias, 8) && aligned_to(dx, 2 * sizeof(T)) &&
                      aligned_to(dz, 2 * sizeof(T));
    if (nv <= 2 * M && even) held(std::integral_constant<bool, !kWhole<V>>());
    else if (nv <= 2 * M) held(std::false_type());
    else
        group_backward_wide_kernel<T><<<dim3(slabs, *parts), kThreads, 0, s>>>(g, d.mean, d.rstd, dy, d.dy_row, dx, dz, partial);
    const int e = launch_end(kKindGroupNormBwd, s);
    return r != SSD_OK ? r : e;
}

template <typename T, int V>
int group_forward_gate(const GroupNormArgs& g, void* y, float* mean, float* rstd, cudaStream_t s) {
    if (g.gate == kGateSilu) return group_forward_of<T, V, kGateSilu>(g, y, mean, rstd, s);
    if (g.gate == kGateAfter) return group_forward_of<T, V, kGateAfter>(g, y, mean, rstd, s);
    if (g.gate == kGateBefore) return group_forward_of<T, V, kGateBefore>(g, y, mean, rstd, s);
    return group_forward_of<T, V, kGateNone>(g, y, mean, rstd, s);
}
template <typename T, int V>
int group_backward_gate(const GroupNormArgs& g, const GroupNormGrads& d, float* partial, int* parts, cudaStream_t s) {
    if (g.gate == kGateSilu) return group_backward_of<T, V, kGateSilu>(g, d, partial, parts, s);
    if (g.gate == kGateAfter) return group_backward_of<T, V, kGateAfter>(g, d, partial, parts, s);
    if (g.gate == kGateBefore) return group_backward_of<T, V, kGateBefore>(g, d, partial, parts, s);
    return group_backward_of<T, V, kGateNone>(g, d, partial, parts, s);
}

template <typename T>
int group_forward_type(const GroupNormArgs& g, void* y, float* mean, float* rstd, cudaStream_t s) {
    if (in_vectors<T>(g) && aligned_to(y, 16)) return group_forward_gate<T, 16 / sizeof(T)>(g, y, mean, rstd, s);
    return group_forward_gate<T, 2>(g, y, mean, rstd, s);
}
template <typename T>
int group_backward_type(const GroupNormArgs& g, const GroupNormGrads& d, float* partial, int* parts, cudaStream_t s) {
    if (in_vectors<T>(g) && d.dy_row % (16 / sizeof(T)) == 0 && aligned_to(d.dy, 16) && aligned_to(d.dx, 16) && aligned_to(d.dz, 16))
        return group_backward_gate<T, 16 / sizeof(T)>(g, d, partial, parts, s);
    return group_backward_gate<T, 2>(g, d, partial, parts, s);
}

}  // namespace
}  // namespace ssd
