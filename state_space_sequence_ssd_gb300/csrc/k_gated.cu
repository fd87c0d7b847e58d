// k_gated.cu -- the gated linear recurrence: one state per channel, decay and input both gated by the token.
//
//   v = sigmoid(r), g = sigmoid(i), u = A v, a = exp(u), s = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + s_t g_t x_t,   y_t = h_t
//
// A scan over composed pairs: a run of tokens takes h to P h + H with P the product of its decays.  A block holds 64
// channels; its eight warps take eight tokens each at once: every warp composes its own run in registers, the pairs go
// through shared memory, and each warp then walks its tokens again from the state in front of them, with the decays and
// inputs that it still holds.  The blocks of a cluster take neighbouring steps of the sequence and give each other their
// pairs through distributed shared memory, so that one pass over the data serves sequences of any length, with as many blocks
// as fill the SMs.  The inputs come through cp.async two steps ahead.
#include "gated.cuh"

namespace ssd {
namespace {

constexpr int kStages = 2;

struct Cluster {
    float4 pair[2][8][32];  // by turn, rank and lane: P and H of two channels
};

template <typename T>
constexpr int forward_smem() {
    return kStages * 3 * kGatedWarps * kGatedPart<T> + 2 * kGatedWarps * 32 * 16 + (int)sizeof(Cluster);
}

// states: (batch, ceil(seqlen / span), channels), the state in front of each span; y, final_state, states may be null.
template <typename T>
__global__ void __launch_bounds__(kGatedThreads, 2)
gated_forward_kernel(GatedArgs g, int ranks, bool vec, bool vecy, T* __restrict__ y, float* __restrict__ final_state,
                     float* __restrict__ states) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = blockIdx.x % ranks, b = blockIdx.y, c0 = blockIdx.x / ranks * kGatedTile, c = c0 + lane * 2;
    const int left = g.channels - c0;
    unsigned char* mine = smem + warp * 3 * kGatedPart<T>;
    constexpr int STAGE = 3 * kGatedWarps * kGatedPart<T>;
    float4* pairs = reinterpret_cast<float4*>(smem + kStages * STAGE);  // [turn][warp][lane]
    Cluster* cl = reinterpret_cast<Cluster*>(pairs + 2 * kGatedWarps * 32);
    const int n = row_length(g.lengths, b, g.seqlen);
    const int steps = ceil_div(n, kGatedSpan * ranks);
    const T* x = static_cast<const T*>(g.x) + b * g.x_batch + c0;
    const T* r = static_cast<const T*>(g.r) + b * g.r_batch + c0;
    const T* i = static_cast<const T*>(g.i) + b * g.i_batch + c0;
    auto fetch = [&](int step) {
        if (step < steps) {
            const int t0 = (step * ranks + rank) * kGatedSpan + warp * kGatedRun;
            unsigned char* to = mine + (step % kStages) * STAGE;
            gated_fetch<T>(to, x, g.x_token, t0, n, left, vec);
            gated_fetch<T>(to + kGatedPart<T>, r, g.r_token, t0, n, left, vec);
            gated_fetch<T>(to + 2 * kGatedPart<T>, i, g.i_token, t0, n, left, vec);
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) fetch(k);
    const bool in0 = c < g.channels, in1 = c + 1 < g.channels;
    const f32x2 A = pk(in0 ? g.A[c] : 0.f, in1 ? g.A[c + 1] : 0.f);
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
    for (int step = 0; step < steps; ++step) {
        const int turn = step & 1, span = step * ranks + rank;
        const int t0 = span * kGatedSpan + warp * kGatedRun;
        const unsigned char* from = mine + (step % kStages) * STAGE;
        copies_wait<kStages - 1>();
        __syncwarp();
        f32x2 a[kGatedRun], bx[kGatedRun], P = pk(1.f, 1.f), H = pk(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kGatedRun; ++k) {
            f32x2 v, gi, w;
            two_gates(exp_neg(gated_at<T>(from + kGatedPart<T>, k)), exp_neg(gated_at<T>(from + 2 * kGatedPart<T>, k)), v, gi);
            decay_terms(mul2(A, v), a[k], w);
            float w0, w1;
            unpk(w, w0, w1);
            bx[k] = mul2(mul2(pk(sqrt_fast(w0), sqrt_fast(w1)), gi), gated_at<T>(from, k));
        }
        if (t0 + kGatedRun > n) {  // tokens past the length keep the state
#pragma unroll
            for (int k = 0; k < kGatedRun; ++k)
                if (t0 + k >= n) {
                    a[k] = pk(1.f, 1.f);
                    bx[k] = pk(0.f, 0.f);
                }
        }
#pragma unroll
        for (int k = 0; k < kGatedRun; ++k) {
            P = mul2(P, a[k]);
            H = fma2(a[k], H, bx[k]);
        }
        __syncwarp();
        fetch(step + kStages);
        {
            const float2 p2 = unpk(P), h2 = unpk(H);
            pairs[(turn * kGatedWarps + warp) * 32 + lane] = make_float4(p2.x, p2.y, h2.x, h2.y);
        }
        __syncthreads();
        float2 start = h;  // in front of this warp's tokens
        if (ranks == 1) {
#pragma unroll
            for (int k = 0; k < kGatedWarps; ++k) {
                const float4 q = pairs[(turn * kGatedWarps + k) * 32 + lane];
                if (k == warp) start = h;
                if (k == 0 && warp == 0 && states != nullptr) keep(span, h);
                h = onward(make_float2(q.x, q.y), h, make_float2(q.z, q.w));
            }
        } else {
            float2 own_p = make_float2(1.f, 1.f), own_h = make_float2(0.f, 0.f), all_p = own_p, all_h = own_h;
#pragma unroll
            for (int k = 0; k < kGatedWarps; ++k) {
                const float4 q = pairs[(turn * kGatedWarps + k) * 32 + lane];
                if (k == warp) {
                    own_p = all_p;
                    own_h = all_h;
                }
                all_h = onward(make_float2(q.x, q.y), all_h, make_float2(q.z, q.w));
                all_p = make_float2(all_p.x * q.x, all_p.y * q.y);
            }
            if (warp < ranks) give((uint32_t)__cvta_generic_to_shared(&cl->pair[turn][rank][lane]), warp, make_float4(all_p.x, all_p.y, all_h.x, all_h.y));
            sm100::cluster_sync();
            for (int k = 0; k < ranks; ++k) {
                const float4 q = cl->pair[turn][k][lane];
                if (k == rank) {
                    if (warp == 0 && states != nullptr && span < kept) keep(span, h);
                    start = onward(own_p, h, own_h);
                }
                h = onward(make_float2(q.x, q.y), h, make_float2(q.z, q.w));
            }
        }
        if (y == nullptr) continue;
        f32x2 hs = pk(start);
        T* o = y + ((int64_t)b * g.seqlen + t0) * g.channels + c;
#pragma unroll
        for (int k = 0; k < kGatedRun; ++k) {
            hs = fma2(a[k], hs, bx[k]);
            if (t0 + k < n) store_vec<T, 2>(o + (int64_t)k * g.channels, Vec<T, 2>::of_pairs({hs}), g.channels - c, vecy);
        }
    }
    copies_wait<0>();
    if (rank == 0 && warp == 0 && final_state != nullptr) {
        float* p = final_state + (int64_t)b * g.channels + c;
        if (in0) p[0] = h.x;
        if (in1) p[1] = h.y;
    }
    if (states != nullptr)
        for (int span = steps * ranks + rank + warp * ranks; span < kept; span += ranks * kGatedWarps) keep(span, h);
    if (y != nullptr)
        for (int t = n + rank * kGatedWarps + warp; t < g.seqlen; t += ranks * kGatedWarps)
            store_vec<T, 2>(y + ((int64_t)b * g.seqlen + t) * g.channels + c, Vec<T, 2>::zero(), g.channels - c, vecy);
    if (ranks > 1) sm100::cluster_sync();  // no block ends while another may still write to its shared memory
}

// ------------------------------------------------------------------ gradient
//
//   lam_t = dy_t + a_{t+1} lam_{t+1}  (dfinal behind the last token)
//   dx = lam s g,   di = lam s x g (1 - g),   dr = q (1 - v),   q = lam (u a h_{t-1} - (u a^2 / s) g x)
//   dA = sum(q) / A,   dinit = a_0 lam_0
//
// The same blocks walk the steps from the last to the first.  The state in front of a step is one that the forward pass kept,
// so that only lam crosses blocks; within the step the pairs of h go forwards and those of lam backwards through
// the same exchange.  u a^2 / s has the limit 0 at u = 0.
template <typename T>
constexpr int backward_smem() {
    return kStages * 4 * kGatedWarps * kGatedPart<T> + 2 * kGatedWarps * 32 * (16 + 8) + (int)sizeof(Cluster);
}

template <typename T>
__global__ void __launch_bounds__(kGatedThreads, 2)
gated_backward_kernel(GatedArgs g, const float* states, const T* __restrict__ dy, const float* __restrict__ dfinal, int ranks, bool vec, bool vecy,
                      T* __restrict__ dx, T* __restrict__ dr, T* __restrict__ di, float* __restrict__ dinit, float* __restrict__ partial) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = blockIdx.x % ranks, b = blockIdx.y, c0 = blockIdx.x / ranks * kGatedTile, c = c0 + lane * 2;
    const int left = g.channels - c0;
    unsigned char* mine = smem + warp * 4 * kGatedPart<T>;
    constexpr int STAGE = 4 * kGatedWarps * kGatedPart<T>;
    float4* pairs = reinterpret_cast<float4*>(smem + kStages * STAGE);          // [turn][warp][lane]: P and H
    float2* ends = reinterpret_cast<float2*>(pairs + 2 * kGatedWarps * 32);     // what lam's run adds
    Cluster* cl = reinterpret_cast<Cluster*>(ends + 2 * kGatedWarps * 32);
    const int n = row_length(g.lengths, b, g.seqlen);
    const int steps = ceil_div(n, kGatedSpan * ranks), kept = ceil_div(g.seqlen, kGatedSpan);
    const T* x = static_cast<const T*>(g.x) + b * g.x_batch + c0;
    const T* r = static_cast<const T*>(g.r) + b * g.r_batch + c0;
    const T* i = static_cast<const T*>(g.i) + b * g.i_batch + c0;
    const T* y = dy + (int64_t)b * g.seqlen * g.channels + c0;
    auto fetch = [&](int step) {
        if (step >= 0) {
            const int t0 = (step * ranks + rank) * kGatedSpan + warp * kGatedRun;
            unsigned char* to = mine + (step % kStages) * STAGE;
            gated_fetch<T>(to, x, g.x_token, t0, n, left, vec);
            gated_fetch<T>(to + kGatedPart<T>, r, g.r_token, t0, n, left, vec);
            gated_fetch<T>(to + 2 * kGatedPart<T>, i, g.i_token, t0, n, left, vec);
            gated_fetch<T>(to + 3 * kGatedPart<T>, y, g.channels, t0, n, left, vec);
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) fetch(steps - 1 - k);
    const bool in0 = c < g.channels, in1 = c + 1 < g.channels;
    const f32x2 A = pk(in0 ? g.A[c] : -1.f, in1 ? g.A[c + 1] : -1.f);
    float2 mu = make_float2(0.f, 0.f);  // the gradient of the state behind the cluster's step
    if (dfinal != nullptr) {
        const float* p = dfinal + (int64_t)b * g.channels + c;
        if (in0) mu.x = p[0];
        if (in1) mu.y = p[1];
    }
    if (states != nullptr && steps == 0) states = nullptr;
    f32x2 dA = pk(0.f, 0.f);
    for (int step = steps - 1; step >= 0; --step) {
        const int turn = step & 1, span = step * ranks + rank;
        const int t0 = span * kGatedSpan + warp * kGatedRun;
        const unsigned char* from = mine + (step % kStages) * STAGE;
        float2 h = make_float2(0.f, 0.f);  // in front of this block's step
        if (span < kept) {
            const float* p = states + ((int64_t)b * kept + span) * g.channels + c;
            if (in0) h.x = p[0];
            if (in1) h.y = p[1];
        }
        copies_wait<kStages - 1>();
        __syncwarp();
        f32x2 a[kGatedRun], er[kGatedRun], ei[kGatedRun], w[kGatedRun], hs[kGatedRun];
        f32x2 P = pk(1.f, 1.f), H = pk(0.f, 0.f), Q = pk(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kGatedRun; ++k) {
            f32x2 v, gi;
            er[k] = exp_neg(gated_at<T>(from + kGatedPart<T>, k));
            ei[k] = exp_neg(gated_at<T>(from + 2 * kGatedPart<T>, k));
            two_gates(er[k], ei[k], v, gi);
            decay_terms(mul2(A, v), a[k], w[k]);
            if (t0 + k >= n) {  // tokens past the length keep the state
                a[k] = pk(1.f, 1.f);
                w[k] = pk(0.f, 0.f);
            }
            float w0, w1;
            unpk(w[k], w0, w1);
            hs[k] = H;  // what this run's tokens in front of k make of a zero state
            H = fma2(a[k], H, mul2(mul2(pk(sqrt_fast(w0), sqrt_fast(w1)), gi), gated_at<T>(from, k)));
            P = mul2(P, a[k]);
        }
#pragma unroll
        for (int k = kGatedRun - 1; k >= 0; --k) Q = mul2(a[k], add2(Q, gated_at<T>(from + 3 * kGatedPart<T>, k)));
        {
            const float2 p2 = unpk(P), h2 = unpk(H);
            pairs[(turn * kGatedWarps + warp) * 32 + lane] = make_float4(p2.x, p2.y, h2.x, h2.y);
            ends[(turn * kGatedWarps + warp) * 32 + lane] = unpk(Q);
        }
        __syncthreads();
        float2 behind = mu, own_p = make_float2(1.f, 1.f), own_q = make_float2(0.f, 0.f), all_p = own_p, all_q = own_q;
#pragma unroll
        for (int k = 0; k < kGatedWarps; ++k)
            if (k < warp) {
                const float4 q = pairs[(turn * kGatedWarps + k) * 32 + lane];
                h = onward(make_float2(q.x, q.y), h, make_float2(q.z, q.w));
            }
#pragma unroll
        for (int k = kGatedWarps - 1; k >= 0; --k) {
            const float4 q = pairs[(turn * kGatedWarps + k) * 32 + lane];
            const float2 e = ends[(turn * kGatedWarps + k) * 32 + lane], p = make_float2(q.x, q.y);
            if (k == warp) {
                own_p = all_p;
                own_q = all_q;
            }
            all_q = onward(p, all_q, e);
            all_p = make_float2(all_p.x * p.x, all_p.y * p.y);
        }
        if (ranks == 1) {
            behind = onward(own_p, mu, own_q);
            mu = onward(all_p, mu, all_q);
        } else {
            if (warp < ranks) give((uint32_t)__cvta_generic_to_shared(&cl->pair[turn][rank][lane]), warp, make_float4(all_p.x, all_p.y, all_q.x, all_q.y));
            sm100::cluster_sync();
            for (int k = ranks - 1; k >= 0; --k) {
                const float4 q = cl->pair[turn][k][lane];
                if (k == rank) behind = onward(own_p, mu, own_q);
                mu = onward(make_float2(q.x, q.y), mu, make_float2(q.z, q.w));
            }
        }
        {  // the states in front of the tokens
            float2 p = make_float2(1.f, 1.f);
#pragma unroll
            for (int k = 0; k < kGatedRun; ++k) {
                hs[k] = pk(onward(p, h, unpk(hs[k])));
                const float2 ak = unpk(a[k]);
                p = make_float2(p.x * ak.x, p.y * ak.y);
            }
        }
        f32x2 m = pk(behind);
        const int64_t o = ((int64_t)b * g.seqlen + t0) * g.channels + c;
#pragma unroll
        for (int k = kGatedRun - 1; k >= 0; --k) {
            const f32x2 xk = gated_at<T>(from, k), lam = add2(m, gated_at<T>(from + 3 * kGatedPart<T>, k));
            f32x2 v, gi, v_rest, g_rest;
            two_gates<true>(er[k], ei[k], v, gi, v_rest, g_rest);
            float w0, w1;
            unpk(w[k], w0, w1);
            const f32x2 rs = pk(w0 < 0x1p-126f ? 0.f : rsqrt_fast(w0), w1 < 0x1p-126f ? 0.f : rsqrt_fast(w1));
            const f32x2 ox = mul2(lam, mul2(mul2(w[k], rs), gi)), oi = mul2(mul2(ox, xk), g_rest);
            // q = lam u a (h - (a / s) g x)
            const f32x2 q = mul2(mul2(lam, mul2(mul2(A, v), a[k])), fma2(mul2(mul2(a[k], rs), mul2(gi, xk)), pk(-1.f, -1.f), hs[k]));
            const f32x2 orr = mul2(q, v_rest);
            m = mul2(a[k], lam);
            if (t0 + k < n) {
                dA = add2(dA, q);
                const int64_t at = o + (int64_t)k * g.channels;
                store_vec<T, 2>(dx + at, Vec<T, 2>::of_pairs({ox}), g.channels - c, vecy);
                store_vec<T, 2>(dr + at, Vec<T, 2>::of_pairs({orr}), g.channels - c, vecy);
                store_vec<T, 2>(di + at, Vec<T, 2>::of_pairs({oi}), g.channels - c, vecy);
            }
        }
        __syncwarp();
        fetch(step - kStages);
    }
    copies_wait<0>();
    if (rank == 0 && warp == 0 && dinit != nullptr) {
        float* p = dinit + (int64_t)b * g.channels + c;
        if (in0) p[0] = mu.x;
        if (in1) p[1] = mu.y;
    }
    for (int t = n + rank * kGatedWarps + warp; t < g.seqlen; t += ranks * kGatedWarps) {
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
        for (int k = 0; k < kGatedWarps; ++k) {
            const float2 e = ends[k * 32 + lane];
            s.x += e.x;
            s.y += e.y;
        }
        float* p = partial + ((int64_t)b * ranks + rank) * g.channels + c;
        if (in0) p[0] = s.x;
        if (in1) p[1] = s.y;
    }
    if (ranks > 1) sm100::cluster_sync();
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
                                                         int* err, bool vec) {
    const int c = (blockIdx.x * 128 + threadIdx.x) * V, b = blockIdx.y;
    if (c >= g.channels) return;
    const int left = g.channels - c;
    const auto x = load_vec<T, V>(static_cast<const T*>(g.x) + b * g.x_batch + c, left, vec);
    const auto r = load_vec<T, V>(static_cast<const T*>(g.r) + b * g.r_batch + c, left, vec);
    const auto i = load_vec<T, V>(static_cast<const T*>(g.i) + b * g.i_batch + c, left, vec);
    const int slot = row_slot(slots, b, nslots, threadIdx.x == 0 ? err : nullptr);
    f32x2 out[(V + 1) / 2];
    float* p = state + (int64_t)(slot < 0 ? 0 : slot) * g.channels + c;
#pragma unroll
    for (int e = 0; e < (V + 1) / 2; ++e) {
        const bool in0 = 2 * e < left && slot >= 0, in1 = 2 * e + 1 < V && 2 * e + 1 < left && slot >= 0;
        const f32x2 A = pk(in0 ? g.A[c + 2 * e] : 0.f, in1 ? g.A[c + 2 * e + 1] : 0.f);
        f32x2 v, gi, a, w;
        two_gates(exp_neg(r.pair(e)), exp_neg(i.pair(e)), v, gi);
        decay_terms(mul2(A, v), a, w);
        float w0, w1;
        unpk(w, w0, w1);
        const f32x2 h = pk(in0 ? p[2 * e] : 0.f, in1 ? p[2 * e + 1] : 0.f);
        out[e] = fma2(a, h, mul2(mul2(pk(sqrt_fast(w0), sqrt_fast(w1)), gi), x.pair(e)));
        const float2 o = unpk(out[e]);
        if (in0) p[2 * e] = o.x;
        if (in1) p[2 * e + 1] = o.y;
        if (slot < 0) out[e] = pk(0.f, 0.f);
    }
    store_vec<T, V>(y + (int64_t)b * g.channels + c, Vec<T, V>::of_pairs(out), left, vec);
}

// Blocks of a cluster, a power of two: enough that about three blocks are there for every SM, none without a step.
int gated_ranks(const GatedArgs& g) {
    const int64_t blocks = (int64_t)ceil_div(g.channels, kGatedTile) * g.batch;
    const int most = ceil_div(g.seqlen, kGatedSpan);
    int k = 1;
    while (k < 8 && 2 * k <= most && blocks * k * 2 <= 3 * kSms) k *= 2;
    return k;
}

template <typename K, typename... Args>
int launch_cluster(K kernel, dim3 grid, int ranks, int smem, cudaStream_t s, Args... args) {
    const int r = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
    if (r != SSD_OK) return r;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kGatedThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ranks;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
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

template <typename T>
int forward_of(const GatedArgs& g, void* y, float* final_state, float* states, cudaStream_t s) {
    const int ranks = gated_ranks(g);
    launch_begin(kKindGated, s);
    const int r = launch_cluster(gated_forward_kernel<T>, dim3(ceil_div(g.channels, kGatedTile) * ranks, g.batch), ranks, forward_smem<T>(), s, g, ranks,
                                 rows_in_vectors<T>(g), g.channels % 2 == 0 && aligned_to(y, 2 * sizeof(T)), static_cast<T*>(y), final_state, states);
    const int e = launch_end(kKindGated, s);
    return r != SSD_OK ? r : e;
}

template <typename T>
int backward_of(const GatedArgs& g, const GatedGrads& d, const float* states, float* partial, cudaStream_t s) {
    const int ranks = gated_ranks(g);
    const bool vecy = g.channels % 2 == 0 && aligned_to(d.dx, 2 * sizeof(T)) && aligned_to(d.dr, 2 * sizeof(T)) && aligned_to(d.di, 2 * sizeof(T));
    launch_begin(kKindGatedBwd, s);
    int r = launch_cluster(gated_backward_kernel<T>, dim3(ceil_div(g.channels, kGatedTile) * ranks, g.batch), ranks, backward_smem<T>(), s, g, states,
                           static_cast<const T*>(d.dy), d.dfinal, ranks, rows_in_vectors<T>(g) && aligned_to(d.dy, 16), vecy, static_cast<T*>(d.dx),
                           static_cast<T*>(d.dr), static_cast<T*>(d.di), d.dinit, partial);
    int e = launch_end(kKindGatedBwd, s);
    r = r != SSD_OK ? r : e;
    if (r != SSD_OK) return r;
    launch_begin(kKindGatedBwd, s);
    launch_dependent(gated_sums_kernel, dim3(ceil_div(g.channels, 32)), dim3(256), 0, s, (const float*)partial, ranks * g.batch, g.channels, g.A, d.dA);
    return launch_end(kKindGatedBwd, s);
}

template <typename T>
int step_of(const GatedArgs& g, float* state, const int* slots, int nslots, void* y, int* err, cudaStream_t s) {
    constexpr int V = 8 / sizeof(T);
    const bool vec = g.channels % V == 0 && g.x_batch % V == 0 && g.r_batch % V == 0 && g.i_batch % V == 0 && aligned_to(g.x, 8) && aligned_to(g.r, 8) &&
                     aligned_to(g.i, 8) && aligned_to(y, 8);
    launch_begin(kKindGatedStep, s);
    gated_step_kernel<T, V><<<dim3(ceil_div(g.channels, 128 * V), g.batch), 128, 0, s>>>(g, state, slots, nslots, static_cast<T*>(y), err, vec);
    return launch_end(kKindGatedStep, s);
}

}  // namespace

size_t gated_states_floats(const GatedArgs& g) { return (size_t)g.batch * ceil_div(g.seqlen, kGatedSpan) * g.channels; }
size_t gated_sums_floats(const GatedArgs& g) { return (size_t)g.batch * gated_ranks(g) * g.channels; }

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
