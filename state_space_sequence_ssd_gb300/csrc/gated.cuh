// gated.cuh -- the gated linear recurrence's terms and the composition of runs of tokens, shared by its kernels.
#pragma once

#include "ops.cuh"
#include "sm100.cuh"

namespace ssd {

// Two channels a lane, 64 a block; eight warps of eight consecutive tokens each, SSD_GATED_SPAN a block and step.
constexpr int kGatedWarps = 8, kGatedRun = 8, kGatedThreads = 32 * kGatedWarps, kGatedTile = 64;
constexpr int kGatedSpan = kGatedWarps * kGatedRun;
static_assert(kGatedSpan == SSD_GATED_SPAN, "a kept state is the one in front of a block's step");

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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

// v = 1 / (1 + er) and g = 1 / (1 + ei), er = e^-r and ei = e^-i.  One reciprocal serves both: 1 / ((1 + er) (1 + ei)) times the
// other's denominator.  Where an exponential passes 2^60 the product could overflow, and a NaN of one gate would reach the
// other: there each has its own.  REST: also 1 - v = er v and 1 - g = ei g, which cancel nothing where v and g are near one.
template <bool REST>
__device__ __forceinline__ void two_gates(f32x2 er, f32x2 ei, f32x2& v, f32x2& g, f32x2& v_rest, f32x2& g_rest) {
    const f32x2 one = pk(1.f, 1.f), p = add2(er, one), q = add2(ei, one);
    float r0, r1, i0, i1, a, b;
    unpk(er, r0, r1);
    unpk(ei, i0, i1);
    if (max_nan(max_nan(r0, r1), max_nan(i0, i1)) <= 0x1p60f) {
        unpk(mul2(p, q), a, b);
        const f32x2 inv = pk(rcp_fast(a), rcp_fast(b));
        v = mul2(q, inv);
        g = mul2(p, inv);
        if (REST) {
            v_rest = mul2(er, v);
            g_rest = mul2(ei, g);
        }
    } else {
        unpk(p, a, b);
        v = pk(rcp_fast(a), rcp_fast(b));
        unpk(q, a, b);
        g = pk(rcp_fast(a), rcp_fast(b));
        if (REST) {  // past 2^60 the rest is one
            unpk(mul2(er, v), a, b);
            v_rest = pk(r0 > 0x1p60f ? 1.f : a, r1 > 0x1p60f ? 1.f : b);
            unpk(mul2(ei, g), a, b);
            g_rest = pk(i0 > 0x1p60f ? 1.f : a, i1 > 0x1p60f ? 1.f : b);
        }
    }
}
__device__ __forceinline__ void two_gates(f32x2 er, f32x2 ei, f32x2& v, f32x2& g) {
    f32x2 none;
    two_gates<false>(er, ei, v, g, none, none);
}

// a = e^u and w = 1 - a^2 for u <= 0.  Near zero 1 - a^2 cancels: there e^u - 1 is Taylor's polynomial of degree 6 (what it
// leaves out is below 2^-24 of it for |u| < 1/4), and w = -(a - 1)(a + 1).  Beyond, e^u is the special function unit's,
// and 1 - a is at least 0.22, so that its error stays below 2^-19.
__device__ __forceinline__ void decay_terms(f32x2 u, f32x2& a, f32x2& w) {
    f32x2 t = fma2(u, pk(1.f / 720, 1.f / 720), pk(1.f / 120, 1.f / 120));
    t = fma2(t, u, pk(1.f / 24, 1.f / 24));
    t = fma2(t, u, pk(1.f / 6, 1.f / 6));
    t = fma2(t, u, pk(0.5f, 0.5f));
    t = fma2(t, u, pk(1.f, 1.f));
    t = mul2(t, u);
    float u0, u1, m0, m1, a0, a1;
    unpk(u, u0, u1);
    unpk(t, m0, m1);
    unpk(add2(t, pk(1.f, 1.f)), a0, a1);
    const float e0 = exp2_fast(u0 * kLog2e), e1 = exp2_fast(u1 * kLog2e);
    const bool near0 = u0 > -0.25f, near1 = u1 > -0.25f;
    a = pk(near0 ? a0 : e0, near1 ? a1 : e1);
    const f32x2 m = pk(near0 ? m0 : e0 - 1.f, near1 ? m1 : e1 - 1.f);
    w = mul2(mul2(m, pk(-1.f, -1.f)), add2(m, pk(2.f, 2.f)));
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

// A warp's part of a step: its kGatedRun rows of the block's channels, one after another in shared memory.
template <typename T>
constexpr int kGatedRow = kGatedTile * (int)sizeof(T);  // bytes of a row
template <typename T>
constexpr int kGatedPart = kGatedRun * kGatedRow<T>;  // of a warp's rows of one tensor

// Copies tokens t0 .. t0 + kGatedRun - 1 of one tensor into the warp's part; tokens from n on and channels past the tensor's
// are zeros.  `p` is the row's first token at channel c0, `left` its channels from there.  vec: whole 16-byte vectors.
template <typename T>
__device__ __forceinline__ void gated_fetch(unsigned char* to, const T* p, int64_t token, int t0, int n, int left, bool vec) {
    constexpr int V = 16 / sizeof(T), PER = kGatedTile / V, ROWS = 32 / PER;
    const int lane = threadIdx.x & 31;
    if (vec) {
        const int c = (lane % PER) * V, r0 = lane / PER;
#pragma unroll
        for (int k = 0; k < kGatedRun / ROWS; ++k) {
            const int r = k * ROWS + r0;
            const bool in = t0 + r < n && c < left;
            copy16(to + r * kGatedRow<T> + c * (int)sizeof(T), in ? p + (t0 + r) * token + c : p, in);
        }
    } else {
        T* s = reinterpret_cast<T*>(to) + lane * 2;
        T v[kGatedRun][2];
#pragma unroll
        for (int r = 0; r < kGatedRun; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                v[r][e] = t0 + r < n && lane * 2 + e < left ? p[(t0 + r) * token + lane * 2 + e] : from_f32<T>(0.f);
#pragma unroll
        for (int r = 0; r < kGatedRun; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[r * kGatedTile + e] = v[r][e];
    }
}
template <typename T>
__device__ __forceinline__ f32x2 gated_at(const unsigned char* part, int r) {
    Vec<T, 2> q;
    const unsigned char* p = part + r * kGatedRow<T> + (threadIdx.x & 31) * 2 * (int)sizeof(T);
    if constexpr (sizeof(T) == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        q.w[0] = u.x;
        q.w[1] = u.y;
    } else {
        q.w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
    return q.pair(0);
}

// One float4 of a lane into the same place of the shared memory of the cluster's block `rank`.
__device__ __forceinline__ void give(uint32_t saddr, uint32_t rank, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(sm100::map_shared_rank(saddr, rank)), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w)
                 : "memory");
}

}  // namespace ssd
