// gated.cuh -- the gated linear recurrence's terms and the composition of runs of tokens, shared by its kernels.
#pragma once

#include "ops.cuh"
#include "sm100.cuh"

namespace ssd {

// Two channels a lane, 64 a block; a block's warps hold SSD_GATED_SPAN consecutive tokens between them.
constexpr int kGatedTile = 64, kGatedSpan = SSD_GATED_SPAN;

constexpr int kGatedRanks = 8;  // blocks of a cluster at most
constexpr int kGatedWait = 61;  // a cluster's wait that gave up, in the device error words

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float sqrt_fast(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rsqrt_fast(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// e^-v of two channels.
__device__ __forceinline__ f32x2 exp_neg(f32x2 v) { return exp2_2(mul2(v, pk(-kLog2e, -kLog2e))); }

// v = 1 / (1 + er) and g = 1 / (1 + ei), er = e^-r and ei = e^-i.  ONE: one reciprocal serves both, 1 / ((1 + er) (1 + ei)) times the
// other's denominator.  The product may then not overflow, nor one of them be a NaN, which would reach the other: `top` is the
// largest product so far, or a NaN, and the values stand where it is at most kShared.
constexpr float kShared = 0x1p120f;
template <bool ONE>
__device__ __forceinline__ void two_gates(f32x2 er, f32x2 ei, f32x2& v, f32x2& g, float& top) {
    const f32x2 one = pk(1.f, 1.f), p = add2(er, one), q = add2(ei, one);
    float a, b;
    if (ONE) {
        unpk(mul2(p, q), a, b);
        top = max_nan(top, a, b);
        const f32x2 inv = pk(rcp_fast(a), rcp_fast(b));
        v = mul2(q, inv);
        g = mul2(p, inv);
    } else {
        unpk(p, a, b);
        v = pk(rcp_fast(a), rcp_fast(b));
        unpk(q, a, b);
        g = pk(rcp_fast(a), rcp_fast(b));
    }
}
template <bool ONE>
__device__ __forceinline__ void two_gates(f32x2 er, f32x2 ei, f32x2& v, f32x2& g) {
    float none = 0.f;
    two_gates<ONE>(er, ei, v, g, none);
}
// 1 - v = er v, which cancels nothing where v is near one; past 2^60 it is one.
template <bool ONE>
__device__ __forceinline__ f32x2 gate_rest(f32x2 er, f32x2 v) {
    if (ONE) return mul2(er, v);
    float r0, r1, a, b;
    unpk(er, r0, r1);
    unpk(mul2(er, v), a, b);
    return pk(r0 > 0x1p60f ? 1.f : a, r1 > 0x1p60f ? 1.f : b);
}
// Whether one reciprocal may serve both gates of all of R tokens.
template <int R>
__device__ __forceinline__ bool gates_share(const f32x2 (&er)[R], const f32x2 (&ei)[R]) {
    float m = 0.f, a, b;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        unpk(er[k], a, b);
        m = max_nan(m, a, b);
        unpk(ei[k], a, b);
        m = max_nan(m, a, b);
    }
    return m <= 0x1p60f;
}

// a = e^u and w = 1 - a^2 for u <= 0.  With n the whole number next to u / ln 2 and f = u - n ln 2, |f| <= ln 2 / 2, e^u - 1 is
// 2^n (e^f - 1) + (2^n - 1).  (e^f - 1) / f is fitted by a polynomial of degree 5 through the Chebyshev expansion (largest error
// 0.42 2^-24, 2.2 with its float32 evaluation).  Near u = 0 n is 0 and nothing cancels: w = -(a - 1)(a + 1) is right to 4 roundings
// and a to 2 there, and within 6 everywhere (samples over [-87, 0]).  Adding 1.5 2^23 rounds to n and leaves it in the low bits,
// from where it goes to the exponent.  In packed arithmetic this takes fewer instructions than the special function unit's
// exponential with a polynomial beside it for small u, and leaves that unit, which the gates keep busy, one call less of five.
// CLAMP: u may be below kDeepest; a is about 2^-126 for all of those.
constexpr float kDeepest = -87.f;
template <bool CLAMP>
__device__ __forceinline__ void decay_terms(f32x2 u, f32x2& a, f32x2& w) {
    if (CLAMP) {
        float u0, u1;
        unpk(u, u0, u1);
        u = pk(max_nan(u0, kDeepest), max_nan(u1, kDeepest));
    }
    const f32x2 t = fma2(u, pk(kLog2e, kLog2e), pk(12582912.f, 12582912.f)), n = add2(t, pk(-12582912.f, -12582912.f));
    const f32x2 f = fma2(n, pk(-0.6931471805599453f, -0.6931471805599453f), u);
    f32x2 p = fma2(f, pk(0.0013933649752289057f, 0.0013933649752289057f), pk(0.00836915522813797f, 0.00836915522813797f));
    p = fma2(p, f, pk(0.04166646674275398f, 0.04166646674275398f));
    p = fma2(p, f, pk(0.16666504740715027f, 0.16666504740715027f));
    p = fma2(p, f, pk(0.5f, 0.5f));
    p = fma2(p, f, pk(1.f, 1.f));
    p = mul2(p, f);
    float t0, t1;
    unpk(t, t0, t1);
    const f32x2 scale = pk(__uint_as_float((__float_as_uint(t0) << 23) + 0x3f800000u), __uint_as_float((__float_as_uint(t1) << 23) + 0x3f800000u));
    const f32x2 m = fma2(p, scale, add2(scale, pk(-1.f, -1.f)));
    a = fma2(p, scale, scale);
    w = mul2(m, fma2(m, pk(-1.f, -1.f), pk(-2.f, -2.f)));
}

// The state h after tokens that multiply it by p and add own.  p may have rounded to zero where no single decay is: an infinite
// state stays infinite then, as it does token by token.
__device__ __forceinline__ float onward(float p, float h, float own) {
    return p == 0.f && fabsf(h) == __int_as_float(0x7f800000) ? h + own : fmaf(p, h, own);
}
__device__ __forceinline__ float2 onward(float2 p, float2 h, float2 own) {
    return make_float2(onward(p.x, h.x, own.x), onward(p.y, h.y, own.y));
}
__device__ __forceinline__ f32x2 pk(float2 v) { return pk(v.x, v.y); }
__device__ __forceinline__ float2 unpk(f32x2 v) {
    float2 r;
    unpk(v, r.x, r.y);
    return r;
}

// h after a run that multiplies it by q.xy and adds q.zw.  SAFE: as above; else a product that rounded to zero may make a NaN
// of an infinity, which the caller looks for (a composition without infinities is an instruction for both channels).
template <bool SAFE>
__device__ __forceinline__ float2 run_after(float2 h, float2 p, float2 own) {
    return SAFE ? onward(p, h, own) : unpk(fma2(pk(p), pk(h), pk(own)));
}
template <bool SAFE>
__device__ __forceinline__ float2 run_after(float2 h, float4 q) {
    return run_after<SAFE>(h, make_float2(q.x, q.y), make_float2(q.z, q.w));
}
__device__ __forceinline__ float2 times(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ bool has_nan(float2 v) { return !(v.x == v.x && v.y == v.y); }

// A warp's R rows (tokens) of one tensor, 64 channels each, on their way through shared memory.  VEC: rows are whole 16-byte vectors,
// and lie there as they are.  Else they are copied in words of four bytes, a word a lane; a row of 16-bit elements that begins in the
// middle of a word lies there shifted by an element, and its words that are not within the tensor's own row are copied
// as the one element that is.
template <typename T, int R, bool VEC>
struct GatedRows {
    static constexpr bool HALF = sizeof(T) == 2;
    static constexpr int PITCH = kGatedTile * (int)sizeof(T) + (VEC || !HALF ? 0 : 4), BYTES = R * PITCH, V = 16 / (int)sizeof(T);
    const T* p;  // VEC: this lane's vector of the row's first token; else that token at the block's first channel
    // 16-bit elements without VEC: whether even and odd tokens' rows begin in the middle of a word, 0 or 1.  (A run begins at an even token.)
    int shift[2];

    __device__ __forceinline__ void begin(const void* tensor, int64_t batch, int64_t token, int c0) {
        p = static_cast<const T*>(tensor) + batch + c0;
        if (VEC) {
            const int lane = threadIdx.x & 31;
            p += lane / (kGatedTile / V) * token + lane % (kGatedTile / V) * V;
        } else if (HALF) {
            shift[0] = (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
            shift[1] = (shift[0] + (int)token) & 1;
        }
    }
    // Tokens t0 .. t0 + R - 1 to `to`; those from n on and channels past the tensor's (`left` from the block's first) are zeros, or,
    // without VEC, not written.
    __device__ __forceinline__ void fetch(unsigned char* to, int64_t token, int t0, int n, int c0, int left) const {
        const int lane = threadIdx.x & 31;
        if constexpr (VEC) {
            constexpr int PER = kGatedTile / V, ROWS = 32 / PER;
            const bool in = lane % PER * V < left;
            const int r0 = lane / PER;
            const T* q = p + t0 * token;
            to += lane * 16;
            if (t0 + R <= n) {
#pragma unroll
                for (int k = 0; k < R / ROWS; ++k, q += ROWS * token) copy16(to + k * 32 * 16, q, in);
            } else {
#pragma unroll
                for (int k = 0; k < R / ROWS; ++k, q += ROWS * token) copy16(to + k * 32 * 16, q, in && t0 + k * ROWS + r0 < n);
            }
        } else {
            const int rows = n - t0 < R ? n - t0 : R;
            const T* q = p + t0 * token;
            if constexpr (HALF) {
                // element e of row r lies at T number e + shift[r & 1] of its place
                const bool even = 2 * lane - shift[0] >= -c0 && 2 * lane - shift[0] + 1 < left;
                const bool odd = 2 * lane - shift[1] >= -c0 && 2 * lane - shift[1] + 1 < left;
                const T *from0 = q + 2 * lane - shift[0], *from1 = q + token + 2 * lane - shift[1];
#pragma unroll
                for (int r = 0; r < R; r += 2, from0 += 2 * token, from1 += 2 * token) {
                    if (even && r < rows) copy4(to + r * PITCH + lane * 4, from0);
                    if (odd && r + 1 < rows) copy4(to + (r + 1) * PITCH + lane * 4, from1);
                }
                // a lane a row: a shifted row's last channel, which begins one more word, and the elements whose word is only half the row's
                if (lane < rows) {
                    const int off = shift[lane & 1], last = left - 1;
                    const T* row = q + lane * token;
                    T* place = reinterpret_cast<T*>(to + lane * PITCH) + off;
                    if (off && left > kGatedTile) copy4(place + kGatedTile - 1, row + kGatedTile - 1);
                    if (off && c0 == 0) place[0] = row[0];
                    if (last < kGatedTile && (last + off) % 2 == 0) place[last] = row[last];
                }
            } else {
                const T* from = q + lane;
                to += lane * 4;
#pragma unroll
                for (int r = 0; r < R; ++r, from += token) {
                    if (lane < left && r < rows) copy4(to + r * PITCH, from);
                    if (lane + 32 < left && r < rows) copy4(to + r * PITCH + 128, from + 32);
                }
            }
        }
    }
    // This lane's two channels of row r.
    __device__ __forceinline__ f32x2 at(const unsigned char* part, int r) const {
        const unsigned char* q = part + r * PITCH + (threadIdx.x & 31) * 2 * (int)sizeof(T);
        Vec<T, 2> v;
        if constexpr (!HALF) {
            const uint2 u = *reinterpret_cast<const uint2*>(q);
            v.w[0] = u.x;
            v.w[1] = u.y;
        } else if constexpr (VEC) {
            v.w[0] = *reinterpret_cast<const uint32_t*>(q);
        } else {
            const T* e = reinterpret_cast<const T*>(q) + shift[r & 1];
            return pk(to_f32<T>(e[0]), to_f32<T>(e[1]));
        }
        return v.pair(0);
    }
};

// The exchange of a cluster's blocks: every step each block gives all of them (itself too) one float4 a lane, with asynchronous stores
// that complete a barrier of the receiver, so that nobody waits for its own stores to global memory, as a cluster barrier's
// release would (2 x 4096 x 4096 of bfloat16: 80 us with one where these took 69).  Two places take turns: a block gives step s + 2 only
// when it has everyone's step s + 1, which they give after they have read step s.  Waits have a limit (Ctl).  A block whose wait
// ran out neither gives nor waits from then on, so that every barrier is armed only behind a phase that completed; the
// others' waits run out in turn.
struct Cluster {
    uint64_t full[2];
    int abort, pad[3];
    // behind it float4 by turn, rank and lane
    __device__ __forceinline__ float4* pair(int turn, int rank, int ranks) {
        return reinterpret_cast<float4*>(this + 1) + (turn * ranks + rank) * 32 + (threadIdx.x & 31);
    }
};
constexpr int cluster_bytes(int ranks) { return (int)sizeof(Cluster) + (ranks > 1 ? 2 * ranks * 32 * (int)sizeof(float4) : 0); }
__device__ __forceinline__ void cluster_begin(Cluster* cl, int ranks) {
    if (ranks == 1) return;
    if (threadIdx.x == 0) {
        cl->abort = 0;
        sm100::mbar_init(&cl->full[0], 1);
        sm100::mbar_init(&cl->full[1], 1);
        sm100::fence_barrier_init();
    }
    sm100::cluster_sync();
}
// Called by one warp: the block's float4 of a step.
__device__ __forceinline__ void cluster_give(Cluster* cl, int step, int rank, int ranks, float4 v, const Ctl& ctl) {
    if (*static_cast<volatile int*>(&cl->abort)) return;  // set in front of the block's last barrier
    const int turn = step & 1, lane = threadIdx.x & 31;
    if (lane == 0 && !(ctl.stall && step == 0)) sm100::mbar_arrive_expect_tx(&cl->full[turn], ranks * 32 * (uint32_t)sizeof(float4));
    const uint32_t place = sm100::smem_u32(cl->pair(turn, rank, ranks)), bar = sm100::smem_u32(&cl->full[turn]);
    for (int k = 0; k < ranks; ++k)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                         sm100::map_shared_rank(place, k)),
                     "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(sm100::map_shared_rank(bar, k))
                     : "memory");
}
__device__ __forceinline__ void cluster_take(Cluster* cl, int step, const Ctl& ctl) {
    sm100::mbar_wait_bounded(&cl->full[step & 1], (step >> 1) & 1, &cl->abort, ctl.err, kGatedWait, ctl.wait_ns);
}
// No block ends while another may still write to its shared memory: all that is given to it has come, and nobody gives more.  Where a
// wait ran out that cannot be waited for; then a millisecond lets the stores on their way arrive.
__device__ __forceinline__ void cluster_end(Cluster* cl, int steps, int ranks, const Ctl& ctl) {
    if (ranks == 1) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        if (*static_cast<volatile int*>(&cl->abort)) {
            const uint64_t t0 = sm100::globaltimer_ns();
            while (sm100::globaltimer_ns() - t0 < 1000000ull) {}
        } else {
            if (steps > 1) sm100::mbar_wait_drain(&cl->full[steps & 1], ((steps - 2) >> 1) & 1, ctl.err, kGatedWait, kDrainNs);
            if (steps > 0) sm100::mbar_wait_drain(&cl->full[(steps - 1) & 1], ((steps - 1) >> 1) & 1, ctl.err, kGatedWait, kDrainNs);
        }
    }
    sm100::cluster_sync();
}

}  // namespace ssd
