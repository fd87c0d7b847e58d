// k_gated.cu -- the gated linear recurrence: one state per channel, decay and input both gated by the token.
//
//   v = sigmoid(r), g = sigmoid(i), u = A v, a = exp(u), s = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + s_t g_t x_t,   y_t = h_t
//
// A scan over composed pairs: a run of tokens takes h to P h + H with P the product of its decays.  A block holds 64 channels, two a
// lane; its warps take 16 consecutive tokens each at once: every warp composes its own run in registers, the pairs go through
// shared memory, and each warp then walks its tokens again from the state in front of them, with the decays and inputs that it
// still holds.  The blocks of a cluster take neighbouring steps of the sequence and give each other their pairs through
// distributed shared memory, so that one pass over the data serves sequences of any length, with as many blocks as fill the SMs.
// The next step's inputs come through cp.async while this step's pairs are exchanged and its outputs written.
//
// 2 x 4096 x 4096 of bfloat16 takes 68 us (4.0 TB/s; the bytes' floor is 40), of float32 85 (6.3 TB/s; 80), 65536 x 2048 of
// bfloat16 294 (158).  With 16-bit elements latency binds: 13 warps an SM, which the registers allow, use 52% of the issue slots, and no
// pipe is full (the multiplier 38%, the special function unit, which gives four results an element, 29%; about 70 instructions a warp and
// token of its 64 channels would issue in 31 us).  Beside that, 256 blocks on 152 SMs leave some with one where others have two
// (2 x 4096 x 4864, 304 blocks, takes 69), and the exchange between blocks, during which nothing else is issued, takes a tenth
// (2 x 4096 x 9728, without clusters, 123: 5.2 TB/s).
// Runs of 8 tokens take 85 us at the first size (more exchange for the work), copies two steps ahead as long as one.
#include <mutex>

#include "gated.cuh"

namespace ssd {
namespace {

constexpr int R = 16;  // consecutive tokens of a warp

// The gradient's blocks of four warps on an SM, and steps of input on their way (see backward_warps).
template <typename T>
constexpr int kBackResident = sizeof(T) == 4 ? 3 : 2;
template <typename T>
constexpr int kBackStages = sizeof(T) == 4 ? 1 : 2;

template <typename T, int W, bool VEC>
int forward_smem(int ranks) {
    return 3 * W * GatedRows<T, R, VEC>::BYTES + 2 * W * 32 * 16 + cluster_bytes(ranks);
}

// The state behind `count` of a block's runs, and the product of their decays, from h in front of them.
template <bool SAFE>
__device__ __forceinline__ void through_runs(const float4* pairs, int count, float2& h, float2& p) {
#pragma unroll 4
    for (int k = 0; k < count; ++k) {
        const float4 q = pairs[k * 32];
        h = run_after<SAFE>(h, q);
        p = times(p, make_float2(q.x, q.y));
    }
}
// What the blocks of a cluster gave: on from h in front of block `first` through the blocks to `last` (exclusive; backwards if it is smaller).
template <bool SAFE>
__device__ __forceinline__ float2 through_blocks(Cluster* cl, int turn, int ranks, int first, int last, float2 h) {
    const int way = last < first ? -1 : 1;
#pragma unroll 2
    for (int k = first; k != last; k += way) h = run_after<SAFE>(h, *cl->pair(turn, k, ranks));
    return h;
}

// states: (batch, ceil(seqlen / span), channels), the state in front of each span; y, final_state, states may be null.
template <typename T, int W, bool VEC>
__global__ void __launch_bounds__(32 * W, 16 / W)
gated_forward_kernel(GatedArgs g, Ctl ctl, int ranks, bool vecy, T* __restrict__ y, float* __restrict__ final_state, float* __restrict__ states) {
    using Rows = GatedRows<T, R, VEC>;
    constexpr int SPAN = W * R, STAGE = 3 * W * Rows::BYTES;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int rank = blockIdx.x % ranks, b = blockIdx.y, c0 = blockIdx.x / ranks * kGatedTile, c = c0 + lane * 2;
    const int left = g.channels - c0;
    unsigned char* mine = smem + warp * 3 * Rows::BYTES;
    float4* pairs = reinterpret_cast<float4*>(smem + STAGE);  // [turn][warp][lane]
    Cluster* cl = reinterpret_cast<Cluster*>(pairs + 2 * W * 32);
    const int n = row_length(g.lengths, b, g.seqlen);
    const int steps = ceil_div(n, SPAN * ranks);
    int ahead = rank * SPAN + warp * R;  // the first token that is not on its way
    Rows x, r, i;
    x.begin(g.x, b * g.x_batch, g.x_token, c0);
    r.begin(g.r, b * g.r_batch, g.r_token, c0);
    i.begin(g.i, b * g.i_batch, g.i_token, c0);
    if (!VEC) {  // what no copy writes is finite
        for (int k = threadIdx.x; k < STAGE / 4; k += 32 * W) reinterpret_cast<uint32_t*>(smem)[k] = 0u;
        __syncthreads();
    }
    auto fetch = [&] {
        if (ahead < n) {
            x.fetch(mine, g.x_token, ahead, n, c0, left);
            r.fetch(mine + Rows::BYTES, g.r_token, ahead, n, c0, left);
            i.fetch(mine + 2 * Rows::BYTES, g.i_token, ahead, n, c0, left);
        }
        ahead += SPAN * ranks;
        copies_commit();
    };
    fetch();
    cluster_begin(cl, ranks);
    const bool in0 = c < g.channels, in1 = c + 1 < g.channels;
    const float A0 = in0 ? g.A[c] : -1.f, A1 = in1 ? g.A[c + 1] : -1.f;
    const f32x2 A = pk(A0, A1);
    const bool shallow = A0 > kDeepest && A1 > kDeepest;  // no decay needs holding (its gate is at most one)
    float2 h = make_float2(0.f, 0.f);  // in front of the cluster's step
    if (g.init != nullptr) {
        const float* p = g.init + (int64_t)b * g.channels + c;
        if (in0) h.x = p[0];
        if (in1) h.y = p[1];
    }
    const int kept = ceil_div(g.seqlen, kGatedSpan);
    auto keep = [&](int span, float2 v) {
        float* p = states + ((int64_t)b * kept + span) * g.channels + c;
        if (in0) p[0] = v.x;
        if (in1) p[1] = v.y;
    };
    int t0 = rank * SPAN + warp * R;
    for (int step = 0; step < steps; ++step, t0 += SPAN * ranks) {
        const int turn = step & 1;
        copies_wait<0>();
        __syncwarp();
        f32x2 a[R], bx[R], P = pk(1.f, 1.f), H = pk(0.f, 0.f);  // a and bx hold the gates' exponentials first
#pragma unroll
        for (int k = 0; k < R; ++k) {
            a[k] = exp_neg(r.at(mine + Rows::BYTES, k));
            bx[k] = exp_neg(i.at(mine + 2 * Rows::BYTES, k));
        }
        auto terms = [&](auto one) {
            constexpr bool ONE = decltype(one)::value;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                f32x2 v, gi, w;
                two_gates<ONE>(a[k], bx[k], v, gi);
                decay_terms<!ONE>(mul2(A, v), a[k], w);
                float w0, w1;
                unpk(w, w0, w1);
                bx[k] = mul2(mul2(pk(sqrt_fast(w0), sqrt_fast(w1)), gi), x.at(mine, k));
                if (!ONE && t0 + k >= n) {  // tokens past the length keep the state
                    a[k] = pk(1.f, 1.f);
                    bx[k] = pk(0.f, 0.f);
                }
            }
        };
        const bool whole = t0 + R <= n;
        if (whole && shallow && gates_share(a, bx)) terms(std::true_type());
        else terms(std::false_type());
#pragma unroll
        for (int k = 0; k < R; ++k) {
            P = mul2(P, a[k]);
            H = fma2(a[k], H, bx[k]);
        }
        __syncwarp();
        fetch();
        {
            const float2 p2 = unpk(P), h2 = unpk(H);
            pairs[(turn * W + warp) * 32 + lane] = make_float4(p2.x, p2.y, h2.x, h2.y);
        }
        __syncthreads();
        const float4* q = pairs + turn * W * 32 + lane;
        auto exchange = [&](auto safe) {  // h in front of this warp's tokens; h becomes the state behind the cluster's step
            constexpr bool SAFE = decltype(safe)::value;
            const float2 zero = make_float2(0.f, 0.f), one = make_float2(1.f, 1.f);
            float2 at = ranks == 1 ? h : zero, p = one;
            through_runs<SAFE>(q, warp, at, p);
            if (ranks == 1) {
                float2 end = at;
                through_runs<SAFE>(q + warp * 32, W - warp, end, p);
                h = end;
                return at;
            }
            const float2 before = through_blocks<SAFE>(cl, turn, ranks, 0, rank, h);
            h = through_blocks<SAFE>(cl, turn, ranks, rank, ranks, before);
            return run_after<SAFE>(before, p, at);
        };
        if (ranks > 1) {
            if (warp == W - 1) {  // the block's runs composed, for the cluster
                float2 end = make_float2(0.f, 0.f), p = make_float2(1.f, 1.f);
                through_runs<false>(q, W, end, p);
                if (has_nan(end)) {
                    end = make_float2(0.f, 0.f), p = make_float2(1.f, 1.f);
                    through_runs<true>(q, W, end, p);
                }
                cluster_give(cl, step, rank, ranks, make_float4(p.x, p.y, end.x, end.y), ctl);
            }
            cluster_take(cl, step, ctl);
        }
        const float2 before = h;
        float2 start = exchange(std::false_type());
        if (has_nan(start) || has_nan(h)) {
            h = before;
            start = exchange(std::true_type());
        }
        if (states != nullptr && warp * R % kGatedSpan == 0 && t0 < g.seqlen) keep(t0 / kGatedSpan, start);
        if (y == nullptr) continue;
        f32x2 hs = pk(start);
        T* to = y + ((int64_t)b * g.seqlen + t0) * g.channels;  // the same for all lanes
        if (whole && vecy) {
            if (in0) {
#pragma unroll
                for (int k = 0; k < R; ++k, to += g.channels) {
                    hs = fma2(a[k], hs, bx[k]);
                    store_vec<T, 2>(to + (uint32_t)c, Vec<T, 2>::of_pairs({hs}), 2, true);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < R; ++k, to += g.channels) {
                hs = fma2(a[k], hs, bx[k]);
                if (t0 + k < n) store_vec<T, 2>(to + (uint32_t)c, Vec<T, 2>::of_pairs({hs}), g.channels - c, vecy);
            }
        }
    }
    copies_wait<0>();
    if (rank == 0 && warp == 0 && final_state != nullptr) {
        float* p = final_state + (int64_t)b * g.channels + c;
        if (in0) p[0] = h.x;
        if (in1) p[1] = h.y;
    }
    if (states != nullptr)
        for (int span = steps * ranks * (SPAN / kGatedSpan) + rank + warp * ranks; span < kept; span += ranks * W) keep(span, h);
    if (y != nullptr)
        for (int t = n + rank * W + warp; t < g.seqlen; t += ranks * W)
            store_vec<T, 2>(y + ((int64_t)b * g.seqlen + t) * g.channels + c, Vec<T, 2>::zero(), g.channels - c, vecy);
    cluster_end(cl, steps, ranks, ctl);
}

// ------------------------------------------------------------------ gradient
//
//   lam_t = dy_t + a_{t+1} lam_{t+1}  (dfinal behind the last token)
//   dx = lam s g,   di = lam s x g (1 - g),   dr = q (1 - v),   q = lam u a (h_{t-1} - (a / s) g x)
//   dA = sum(q) / A,   dinit = a_0 lam_0
//
// The same blocks walk the steps from the last to the first.  The state in front of a step is one that the forward pass kept,
// so that only lam crosses blocks; within the step the pairs of h go forwards and those of lam backwards through
// the same exchange.  u a / s has the limit 0 at u = 0.
template <typename T, int W, int STAGES, bool VEC>
int backward_smem(int ranks) {
    return STAGES * 4 * W * GatedRows<T, R, VEC>::BYTES + 2 * W * 32 * (16 + 8) + cluster_bytes(ranks);
}

// As through_runs, for lam: from the last run to the first.
template <bool SAFE>
__device__ __forceinline__ void back_through_runs(const float4* pairs, const float2* ends, int from, int to, float2& mu, float2& p) {
#pragma unroll 4
    for (int k = from; k > to; --k) {
        const float2 q = *reinterpret_cast<const float2*>(&pairs[k * 32]);
        mu = run_after<SAFE>(mu, q, ends[k * 32]);
        p = times(p, q);
    }
}

template <typename T, int W, int STAGES, bool VEC>
__global__ void __launch_bounds__(32 * W, W == 4 ? kBackResident<T> : 1)
gated_backward_kernel(GatedArgs g, const float* states, const T* __restrict__ dy, const float* __restrict__ dfinal, Ctl ctl, int ranks, bool vecy,
                      T* __restrict__ dx, T* __restrict__ dr, T* __restrict__ di, float* __restrict__ dinit, float* __restrict__ partial) {
    using Rows = GatedRows<T, R, VEC>;
    constexpr bool FIRST = sizeof(T) == 4;
    constexpr int SPAN = W * R, STAGE = 4 * W * Rows::BYTES;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int rank = blockIdx.x % ranks, b = blockIdx.y, c0 = blockIdx.x / ranks * kGatedTile, c = c0 + lane * 2;
    const int left = g.channels - c0;
    unsigned char* mine = smem + warp * 4 * Rows::BYTES;
    float4* pairs = reinterpret_cast<float4*>(smem + STAGES * STAGE);  // [turn][warp][lane]: P and H
    float2* ends = reinterpret_cast<float2*>(pairs + 2 * W * 32);       // what lam's run adds
    Cluster* cl = reinterpret_cast<Cluster*>(ends + 2 * W * 32);
    const int n = row_length(g.lengths, b, g.seqlen);
    const int steps = ceil_div(n, SPAN * ranks), kept = ceil_div(g.seqlen, kGatedSpan);
    int t0 = ((steps - 1) * ranks + rank) * SPAN + warp * R, ahead = t0;
    Rows x, r, i, gy;
    x.begin(g.x, b * g.x_batch, g.x_token, c0);
    r.begin(g.r, b * g.r_batch, g.r_token, c0);
    i.begin(g.i, b * g.i_batch, g.i_token, c0);
    gy.begin(dy, (int64_t)b * g.seqlen * g.channels, g.channels, c0);
    if (!VEC) {  // what no copy writes is finite
        for (int k = threadIdx.x; k < STAGES * STAGE / 4; k += 32 * W) reinterpret_cast<uint32_t*>(smem)[k] = 0u;
        __syncthreads();
    }
    auto fetch = [&](int stage) {
        unsigned char* to = mine + stage * STAGE;
        if (ahead >= 0) {
            x.fetch(to, g.x_token, ahead, n, c0, left);
            r.fetch(to + Rows::BYTES, g.r_token, ahead, n, c0, left);
            i.fetch(to + 2 * Rows::BYTES, g.i_token, ahead, n, c0, left);
            gy.fetch(to + 3 * Rows::BYTES, g.channels, ahead, n, c0, left);
        }
        ahead -= SPAN * ranks;
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < STAGES; ++k) fetch(k);
    cluster_begin(cl, ranks);
    const bool in0 = c < g.channels, in1 = c + 1 < g.channels;
    const float A0 = in0 ? g.A[c] : -1.f, A1 = in1 ? g.A[c + 1] : -1.f;
    const f32x2 A = pk(A0, A1);
    const bool shallow = A0 > kDeepest && A1 > kDeepest;  // no decay needs holding (its gate is at most one)
    float2 mu = make_float2(0.f, 0.f);  // the gradient of the state behind the cluster's step
    if (dfinal != nullptr) {
        const float* p = dfinal + (int64_t)b * g.channels + c;
        if (in0) mu.x = p[0];
        if (in1) mu.y = p[1];
    }
    auto kept_state = [&](int span) {  // in front of this block's tokens
        float2 v = make_float2(0.f, 0.f);
        const int at = span * (SPAN / kGatedSpan);
        if (at >= 0 && at < kept) {
            const float* p = states + ((int64_t)b * kept + at) * g.channels + c;
            if (in0) v.x = p[0];
            if (in1) v.y = p[1];
        }
        return v;
    };
    float2 next = kept_state((steps - 1) * ranks + rank);
    f32x2 dA = pk(0.f, 0.f);
    for (int step = 0; step < steps; ++step, t0 -= SPAN * ranks) {
        const int turn = step & 1, span = (steps - 1 - step) * ranks + rank;
        const unsigned char* from = mine + (step % STAGES) * STAGE;
        const float2 before = next;
        copies_wait<STAGES - 1>();
        __syncwarp();
        f32x2 a[R], w[R], hs[R];
        f32x2 P = pk(1.f, 1.f), H = pk(0.f, 0.f), Q = pk(0.f, 0.f);
        const bool whole = t0 + R <= n;
        // VEC: x and dy are zero past the length already
        auto x_at = [&](int k) { return VEC || whole || t0 + k < n ? x.at(from, k) : pk(0.f, 0.f); };
        auto dy_at = [&](int k) { return VEC || whole || t0 + k < n ? gy.at(from + 3 * Rows::BYTES, k) : pk(0.f, 0.f); };
        float top = 0.f;
        auto terms = [&](auto one) {
            constexpr bool ONE = decltype(one)::value;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                f32x2 v, gi;
                if (FIRST) two_gates<ONE>(a[k], w[k], v, gi);
                else two_gates<ONE>(exp_neg(r.at(from + Rows::BYTES, k)), exp_neg(i.at(from + 2 * Rows::BYTES, k)), v, gi, top);
                decay_terms<!ONE>(mul2(A, v), a[k], w[k]);
                if (!ONE && t0 + k >= n) {  // tokens past the length keep the state
                    a[k] = pk(1.f, 1.f);
                    w[k] = pk(0.f, 0.f);
                }
                float w0, w1;
                unpk(w[k], w0, w1);
                hs[k] = H;  // what this run's tokens in front of k make of a zero state
                H = fma2(a[k], H, mul2(mul2(pk(sqrt_fast(w0), sqrt_fast(w1)), gi), x_at(k)));
                P = mul2(P, a[k]);
            }
        };
        bool share = false;
        if (FIRST) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                a[k] = exp_neg(r.at(from + Rows::BYTES, k));
                w[k] = exp_neg(i.at(from + 2 * Rows::BYTES, k));
            }
            share = whole && shallow && gates_share(a, w);
            if (share) terms(std::true_type());
        } else if (whole && shallow) {
            terms(std::true_type());
            share = top <= kShared;
        }
        if (!share) {
            P = pk(1.f, 1.f);
            H = pk(0.f, 0.f);
            terms(std::false_type());
        }
#pragma unroll
        for (int k = R - 1; k >= 0; --k) Q = mul2(a[k], add2(Q, dy_at(k)));
        {
            const float2 p2 = unpk(P), h2 = unpk(H);
            pairs[(turn * W + warp) * 32 + lane] = make_float4(p2.x, p2.y, h2.x, h2.y);
            ends[(turn * W + warp) * 32 + lane] = unpk(Q);
        }
        __syncthreads();
        const float4* pq = pairs + turn * W * 32 + lane;
        const float2* eq = ends + turn * W * 32 + lane;
        if (ranks > 1) {
            if (warp == 0) {
                float2 all = make_float2(0.f, 0.f), p = make_float2(1.f, 1.f);
                back_through_runs<false>(pq, eq, W - 1, -1, all, p);
                if (has_nan(all)) {
                    all = make_float2(0.f, 0.f), p = make_float2(1.f, 1.f);
                    back_through_runs<true>(pq, eq, W - 1, -1, all, p);
                }
                cluster_give(cl, step, rank, ranks, make_float4(p.x, p.y, all.x, all.y), ctl);
            }
        }
        float2 h, behind;  // the state in front of this warp's tokens, the gradient of the one behind them
        auto exchange = [&](auto safe) {
            constexpr bool SAFE = decltype(safe)::value;
            const float2 zero = make_float2(0.f, 0.f);
            float2 p = make_float2(1.f, 1.f), own_p = p, own = ranks == 1 ? mu : zero;
            h = before;
            through_runs<SAFE>(pq, warp, h, p);
            back_through_runs<SAFE>(pq, eq, W - 1, warp, own, own_p);
            if (ranks == 1) {
                behind = mu = own;
                back_through_runs<SAFE>(pq, eq, warp, -1, mu, own_p);
            } else {
                const float2 from_others = through_blocks<SAFE>(cl, turn, ranks, ranks - 1, rank, mu);
                mu = through_blocks<SAFE>(cl, turn, ranks, rank, -1, from_others);
                behind = run_after<SAFE>(from_others, own_p, own);
            }
        };
        next = kept_state(span - ranks);
        if (ranks > 1) cluster_take(cl, step, ctl);
        const float2 mu0 = mu;
        exchange(std::false_type());
        if (has_nan(h) || has_nan(behind) || has_nan(mu)) {
            mu = mu0;
            exchange(std::true_type());
        }
        {  // the states in front of the tokens
            f32x2 p = pk(1.f, 1.f);
            const f32x2 h2 = pk(h);
            if (fabsf(h.x) < __int_as_float(0x7f800000) && fabsf(h.y) < __int_as_float(0x7f800000)) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    hs[k] = fma2(p, h2, hs[k]);
                    p = mul2(p, a[k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    hs[k] = pk(onward(unpk(p), h, unpk(hs[k])));
                    p = mul2(p, a[k]);
                }
            }
        }
        f32x2 m = pk(behind);
        auto gradients = [&](auto one, auto packed) {
            constexpr bool ONE = decltype(one)::value, PACKED = decltype(packed)::value;
            int64_t at = ((int64_t)b * g.seqlen + t0 + R - 1) * g.channels;  // the same for all lanes
#pragma unroll
            for (int k = R - 1; k >= 0; --k, at -= g.channels) {
                const f32x2 xk = x_at(k), lam = add2(m, dy_at(k));
                f32x2 v, gi;
                const f32x2 er = exp_neg(r.at(from + Rows::BYTES, k)), ei = exp_neg(i.at(from + 2 * Rows::BYTES, k));
                two_gates<ONE>(er, ei, v, gi);
                float w0, w1;
                unpk(w[k], w0, w1);
                const f32x2 rs = pk(rsqrt_fast(fmaxf(w0, 0x1p-126f)), rsqrt_fast(fmaxf(w1, 0x1p-126f)));  // s = w rs is 0 at w = 0
                const f32x2 gx = mul2(lam, mul2(mul2(w[k], rs), gi)), gi_x = mul2(gi, xk);
                const f32x2 q = mul2(mul2(lam, mul2(mul2(A, v), a[k])), fma2(mul2(mul2(a[k], rs), gi_x), pk(-1.f, -1.f), hs[k]));
                m = mul2(a[k], lam);
                const f32x2 gr = mul2(q, gate_rest<ONE>(er, v)), gi2 = mul2(mul2(gx, xk), gate_rest<ONE>(ei, gi));
                if (ONE && PACKED) {
                    dA = add2(dA, q);
                    if (in0) {
                        store_vec<T, 2>(dx + at + (uint32_t)c, Vec<T, 2>::of_pairs({gx}), 2, true);
                        store_vec<T, 2>(dr + at + (uint32_t)c, Vec<T, 2>::of_pairs({gr}), 2, true);
                        store_vec<T, 2>(di + at + (uint32_t)c, Vec<T, 2>::of_pairs({gi2}), 2, true);
                    }
                } else if (ONE || t0 + k < n) {
                    dA = add2(dA, q);
                    const bool whole_pairs = !ONE && vecy;  // ONE without PACKED: they are not
                    store_vec<T, 2>(dx + at + (uint32_t)c, Vec<T, 2>::of_pairs({gx}), g.channels - c, whole_pairs);
                    store_vec<T, 2>(dr + at + (uint32_t)c, Vec<T, 2>::of_pairs({gr}), g.channels - c, whole_pairs);
                    store_vec<T, 2>(di + at + (uint32_t)c, Vec<T, 2>::of_pairs({gi2}), g.channels - c, whole_pairs);
                }
            }
        };
        if (share && vecy) gradients(std::true_type(), std::true_type());
        else if (!VEC && share) gradients(std::true_type(), std::false_type());
        else gradients(std::false_type(), std::false_type());
        __syncwarp();
        fetch(step % STAGES);
    }
    copies_wait<0>();
    if (rank == 0 && warp == 0 && dinit != nullptr) {
        float* p = dinit + (int64_t)b * g.channels + c;
        if (in0) p[0] = mu.x;
        if (in1) p[1] = mu.y;
    }
    for (int t = n + rank * W + warp; t < g.seqlen; t += ranks * W) {
        const int64_t at = ((int64_t)b * g.seqlen + t) * g.channels + c;
        store_vec<T, 2>(dx + at, Vec<T, 2>::zero(), g.channels - c, vecy);
        store_vec<T, 2>(dr + at, Vec<T, 2>::zero(), g.channels - c, vecy);
        store_vec<T, 2>(di + at, Vec<T, 2>::zero(), g.channels - c, vecy);
    }
    __syncthreads();
    ends[warp * 32 + lane] = unpk(dA);
    __syncthreads();
    if (warp == 0) {
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float2 e = ends[k * 32 + lane];
            s.x += e.x;
            s.y += e.y;
        }
        float* p = partial + ((int64_t)b * ranks + rank) * g.channels + c;
        if (in0) p[0] = s.x;
        if (in1) p[1] = s.y;
    }
    cluster_end(cl, steps, ranks, ctl);
}

// dA: the blocks' sums of q, added in a fixed order, over A.  (`partial` is written while this kernel may already run.)
__global__ void __launch_bounds__(256) gated_sums_kernel(const float* partial, int parts, int channels, const float* __restrict__ A,
                                                         float* __restrict__ dA) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    grid_dep_wait();
    float s = 0.f;
    if (c < channels)
        for (int k = warp; k < parts; k += 8) s += partial[(int64_t)k * channels + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= channels) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += part[k][lane];
    dA[c] = s / A[c];
}

// ------------------------------------------------------------------ one token
template <typename T, int V>
__global__ void __launch_bounds__(128) gated_step_kernel(GatedArgs g, float* state, const int* __restrict__ slots, int nslots, T* __restrict__ y,
                                                         int* err, bool vec, bool vecs) {
    const int c = (blockIdx.x * 128 + threadIdx.x) * V, b = blockIdx.y;
    if (c >= g.channels) return;
    const int left = g.channels - c;
    const auto x = load_vec<T, V>(static_cast<const T*>(g.x) + b * g.x_batch + c, left, vec);
    const auto r = load_vec<T, V>(static_cast<const T*>(g.r) + b * g.r_batch + c, left, vec);
    const auto i = load_vec<T, V>(static_cast<const T*>(g.i) + b * g.i_batch + c, left, vec);
    const int slot = row_slot(slots, b, nslots, threadIdx.x == 0 ? err : nullptr);
    static_assert(V % 2 == 0, "whole pairs");
    float* p = state + (int64_t)(slot < 0 ? 0 : slot) * g.channels + c;
    const auto A = load_vec<float, V>(g.A + c, left, vecs);
    const auto h = load_vec<float, V, true>(p, slot < 0 ? 0 : left, vecs);
    f32x2 out[V / 2];
    float top = 0.f;
    auto token = [&](auto one) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            f32x2 v, gi, a, w;
            two_gates<decltype(one)::value>(exp_neg(r.pair(e)), exp_neg(i.pair(e)), v, gi, top);
            decay_terms<true>(mul2(A.pair(e), v), a, w);
            float w0, w1;
            unpk(w, w0, w1);
            out[e] = fma2(a, h.pair(e), mul2(mul2(pk(sqrt_fast(w0), sqrt_fast(w1)), gi), x.pair(e)));
        }
    };
    token(std::true_type());
    if (!(top <= kShared)) token(std::false_type());
    if (slot >= 0) store_vec<float, V>(p, Vec<float, V>::of_pairs(out), left, vecs);
    if (slot < 0) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) out[e] = pk(0.f, 0.f);
    }
    store_vec<T, V>(y + (int64_t)b * g.channels + c, Vec<T, V>::of_pairs(out), left, vec);
}

cudaLaunchConfig_t cluster_launch(dim3 grid, int threads, int ranks, int smem, cudaStream_t s, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = ranks;
    attr->val.clusterDim.y = 1;
    attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Clusters of `ranks` blocks that the device holds at once; asked for once per kernel, size and device.
template <typename K>
int cluster_room(K kernel, int threads, int ranks, int smem) {
    struct Known {
        const void* kernel;
        int device, ranks, room;
    };
    static std::mutex mu;
    static Known known[256];  // of one signature: its types, warps and kinds of rows, by sizes and devices; asked for again where it is full
    static int count = 0;
    const void* k = reinterpret_cast<const void*>(kernel);
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || ensure_smem_limit(k, 227 * 1024) != SSD_OK) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < count; ++i)
        if (known[i].kernel == k && known[i].device == device && known[i].ranks == ranks) return known[i].room;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = cluster_launch(dim3(ranks), threads, ranks, smem, nullptr, &attr);
    int room = 0;
    if (cudaOccupancyMaxActiveClusters(&room, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        room = 0;
    }
    if (count < 256) known[count++] = {k, device, ranks, room};
    return room;
}

// Blocks of a cluster: the most, none without a step, with which all clusters run at once.  (They need room within one part of the device
// each, so that fewer fit than blocks do: 1 x 4096 x 4864 of bfloat16 takes 57 us in 76 clusters of four, two of which wait for a second
// turn, and 50 in clusters of three, its gradient 123 and 80.)
template <typename K>
int gated_ranks(K kernel, const GatedArgs& g, int warps, int (*smem)(int)) {
    const int64_t blocks = (int64_t)ceil_div(g.channels, kGatedTile) * g.batch;
    const int most = ceil_div(g.seqlen, warps * R);
    for (int k = most < kGatedRanks ? most : kGatedRanks; k > 1; --k)
        if (blocks <= 4 * kSms / k && blocks <= cluster_room(kernel, 32 * warps, k, smem(k))) return k;
    return 1;
}

template <typename K, typename... Args>
int launch_cluster(K kernel, dim3 grid, int threads, int ranks, int smem, cudaStream_t s, Args... args) {
    const int r = ensure_smem_limit(reinterpret_cast<const void*>(kernel), 227 * 1024);
    if (r != SSD_OK) return r;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = cluster_launch(grid, threads, ranks, smem, s, &attr);
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// Whether every token's row is whole 16-byte vectors from the tensor's first channel on.
template <typename T>
bool rows_in_vectors(const GatedArgs& g) {
    constexpr int V = 16 / sizeof(T);
    for (int64_t v : {g.x_batch, g.x_token, g.r_batch, g.r_token, g.i_batch, g.i_token, (int64_t)g.channels})
        if (v % V != 0) return false;
    return aligned_to(g.x, 16) && aligned_to(g.r, 16) && aligned_to(g.i, 16);
}

template <typename T, int W, bool VEC>
int forward_rows(const GatedArgs& g, int ranks, void* y, float* final_state, float* states, cudaStream_t s) {
    launch_begin(kKindGated, s);
    const int r = launch_cluster(gated_forward_kernel<T, W, VEC>, dim3(ceil_div(g.channels, kGatedTile) * ranks, g.batch), 32 * W, ranks,
                                 forward_smem<T, W, VEC>(ranks), s, g, wait_control(kKindGated), ranks,
                                 g.channels % 2 == 0 && aligned_to(y, 2 * sizeof(T)), static_cast<T*>(y), final_state, states);
    const int e = launch_end(kKindGated, s);
    return r != SSD_OK ? r : e;
}
// Eight warps a block; four, and so more blocks, where one step of theirs holds the rows (512 tokens of 256 channels of bfloat16: 5.1 us with
// four, 5.7 with eight; 1024: 7.3 and 6.0; 2 x 4096 of 4096: 71 and 68; 65536 of 2048: 324 and 299).
template <typename T, bool VEC>
int forward_warps(const GatedArgs& g, void* y, float* final_state, float* states, cudaStream_t s) {
    if (g.seqlen <= 4 * R * kGatedRanks) {
        const int four = gated_ranks(gated_forward_kernel<T, 4, VEC>, g, 4, forward_smem<T, 4, VEC>);
        if (four * 4 * R >= g.seqlen) return forward_rows<T, 4, VEC>(g, four, y, final_state, states, s);
    }
    return forward_rows<T, 8, VEC>(g, gated_ranks(gated_forward_kernel<T, 8, VEC>, g, 8, forward_smem<T, 8, VEC>), y, final_state, states, s);
}
template <typename T>
int forward_of(const GatedArgs& g, void* y, float* final_state, float* states, cudaStream_t s) {
    return rows_in_vectors<T>(g) ? forward_warps<T, true>(g, y, final_state, states, s) : forward_warps<T, false>(g, y, final_state, states, s);
}

template <typename T, int W, bool VEC>
int backward_rows(const GatedArgs& g, int ranks, const GatedGrads& d, const float* states, float* partial, cudaStream_t s) {
    constexpr int S = kBackStages<T>;
    const bool vecy = g.channels % 2 == 0 && aligned_to(d.dx, 2 * sizeof(T)) && aligned_to(d.dr, 2 * sizeof(T)) && aligned_to(d.di, 2 * sizeof(T));
    launch_begin(kKindGatedBwd, s);
    int r = launch_cluster(gated_backward_kernel<T, W, S, VEC>, dim3(ceil_div(g.channels, kGatedTile) * ranks, g.batch), 32 * W, ranks,
                           backward_smem<T, W, S, VEC>(ranks), s, g, states, static_cast<const T*>(d.dy), d.dfinal, wait_control(kKindGatedBwd), ranks,
                           vecy, static_cast<T*>(d.dx), static_cast<T*>(d.dr), static_cast<T*>(d.di), d.dinit, partial);
    const int e = launch_end(kKindGatedBwd, s);
    r = r != SSD_OK ? r : e;
    if (r != SSD_OK) return r;
    launch_begin(kKindGatedBwd, s);
    launch_dependent(gated_sums_kernel, dim3(ceil_div(g.channels, 32)), dim3(256), 0, s, (const float*)partial, ranks * g.batch, g.channels, g.A, d.dA);
    return launch_end(kKindGatedBwd, s);
}
// Four warps: with 16-bit tensors two blocks an SM, with up to 255 registers a thread, and two steps of input on their way; three
// with 168 registers, which a 32-bit type's single step of input leaves room for, take 146 us where these take 139 (2 x 4096 x 4096 of
// bfloat16), and 169 where two take 199 (float32).  Eight warps where their clusters, of one block an SM, take in more tokens a step
// (4096 tokens of 96 channels of bfloat16: 35.6 us with four, 22.9 with eight; 2048 of 256 20.0 and 13.7; 2 x 4096 of 512, in clusters of
// six, 37.9 and 32.9; without clusters 8 x 4096 of 4096 474 and 511), and rows take more than one.
template <typename T, bool VEC>
int backward_warps(const GatedArgs& g, const GatedGrads& d, const float* states, float* partial, cudaStream_t s) {
    constexpr int S = kBackStages<T>;
    const int four = gated_ranks(gated_backward_kernel<T, 4, S, VEC>, g, 4, backward_smem<T, 4, S, VEC>);
    if (g.seqlen > four * 4 * R) {
        const int eight = gated_ranks(gated_backward_kernel<T, 8, S, VEC>, g, 8, backward_smem<T, 8, S, VEC>);
        if (eight > 1 && 2 * eight > four) return backward_rows<T, 8, VEC>(g, eight, d, states, partial, s);
    }
    return backward_rows<T, 4, VEC>(g, four, d, states, partial, s);
}
template <typename T>
int backward_of(const GatedArgs& g, const GatedGrads& d, const float* states, float* partial, cudaStream_t s) {
    return rows_in_vectors<T>(g) && aligned_to(d.dy, 16) ? backward_warps<T, true>(g, d, states, partial, s) : backward_warps<T, false>(g, d, states, partial, s);
}

template <typename T>
int step_of(const GatedArgs& g, float* state, const int* slots, int nslots, void* y, int* err, cudaStream_t s) {
    constexpr int V = 8 / sizeof(T);
    const bool vec = g.channels % V == 0 && g.x_batch % V == 0 && g.r_batch % V == 0 && g.i_batch % V == 0 && aligned_to(g.x, 8) && aligned_to(g.r, 8) &&
                     aligned_to(g.i, 8) && aligned_to(y, 8), vecs = g.channels % V == 0 && aligned_to(state, 4 * V) && aligned_to(g.A, 4 * V);
    launch_begin(kKindGatedStep, s);
    gated_step_kernel<T, V><<<dim3(ceil_div(g.channels, 128 * V), g.batch), 128, 0, s>>>(g, state, slots, nslots, static_cast<T*>(y), err, vec, vecs);
    return launch_end(kKindGatedStep, s);
}

}  // namespace

size_t gated_states_floats(const GatedArgs& g) { return (size_t)g.batch * ceil_div(g.seqlen, kGatedSpan) * g.channels; }
size_t gated_sums_floats(const GatedArgs& g) { return (size_t)g.batch * kGatedRanks * g.channels; }

int launch_gated_forward(const GatedArgs& g, void* y, float* final_state, float* states, cudaStream_t s) {
    if (g.dtype == SSD_BF16) return forward_of<__nv_bfloat16>(g, y, final_state, states, s);
    if (g.dtype == SSD_F16) return forward_of<__half>(g, y, final_state, states, s);
    return forward_of<float>(g, y, final_state, states, s);
}

int launch_gated_backward(const GatedArgs& g, const GatedGrads& d, const float* states, float* partial, cudaStream_t s) {
    if (g.dtype == SSD_BF16) return backward_of<__nv_bfloat16>(g, d, states, partial, s);
    if (g.dtype == SSD_F16) return backward_of<__half>(g, d, states, partial, s);
    return backward_of<float>(g, d, states, partial, s);
}

int launch_gated_step(const GatedArgs& g, float* state, const int* slots, int nslots, void* y, int* err, cudaStream_t s) {
    if (g.dtype == SSD_BF16) return step_of<__nv_bfloat16>(g, state, slots, nslots, y, err, s);
    if (g.dtype == SSD_F16) return step_of<__half>(g, state, slots, nslots, y, err, s);
    return step_of<float>(g, state, slots, nslots, y, err, s);
}

}  // namespace ssd
