// norm.cuh -- what the norms' kernels share (k_norm.cu, group_norm.cuh): sums over the threads of a row, loads of weights, and how
// many threads a row gets.
#pragma once

#include "ops.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;  // of a norm's block

// Sums of two values over the `lanes` threads of one row (a power of two; at most kThreads).  Every thread of the
// block calls it.  buf holds a pair per warp; calls that follow one another alternate between two of them, so that
// one barrier a call is enough.
__device__ __forceinline__ float2 row_sums(float2 v, int lanes, float2* buf) {
    if (lanes >= 32) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
    } else {
        for (int o = lanes / 2; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
    }
    if (lanes <= 32) return v;
    const int warp = threadIdx.x >> 5, per = lanes >> 5;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
    for (int i = 0; i < per; ++i) {
        const float2 q = buf[(warp / per) * per + i];
        v.x += q.x;
        v.y += q.y;
    }
    return v;
}
__device__ __forceinline__ float row_sum(float v, int lanes, float2* buf) { return row_sums(make_float2(v, 0.f), lanes, buf).x; }

// The mean of n values from their sum, inv = 1 / n rounded: a plain product is off by up to a unit and a half, which would shift the whole
// group, times rstd; with inv's own error put back the result is the rounded quotient.  An infinite sum stays one.
__device__ __forceinline__ float mean_of(float sum, int n, float inv) {
    const float low = fmaf(-inv, (float)n, 1.f) * inv;
    return fmaf(sum, inv, fminf(fmaxf(sum, -3.4028235e38f), 3.4028235e38f) * low);
}

// Elements 2 i and 2 i + 1 of a vector plus c.  16-bit elements are widened by the addition itself, an instruction each instead of one
// each and a packed addition (8192 x 4096 of float16 in 2 groups, silu of the output, gradient: 72 us; widened first 76).
template <typename T, int V>
__device__ __forceinline__ f32x2 pair_plus(const Vec<T, V>& v, int i, float c) {
    if constexpr (sizeof(T) == 4 || V == 1) {
        return add2(v.pair(i), pk(c, c));
    } else {
        float lo, hi;
        if constexpr (std::is_same<T, __half>::value)
            asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\nadd.rn.f32.f16 %0, l, %3;\nadd.rn.f32.f16 %1, h, %3;\n}" : "=f"(lo), "=f"(hi) : "r"(v.w[i]), "f"(c));
        else
            asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\nadd.rn.f32.bf16 %0, l, %3;\nadd.rn.f32.bf16 %1, h, %3;\n}" : "=f"(lo), "=f"(hi) : "r"(v.w[i]), "f"(c));
        return pk(lo, hi);
    }
}

// V columns of a float32 row from column c on, as pairs (a null row: `otherwise`).  `vec`: 16-byte aligned groups of four.
template <int V>
__device__ __forceinline__ void load_columns(const float* p, int c, int width, bool vec, float otherwise,
                                             f32x2 (&o)[(V + 1) / 2]) {
    if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < (V + 1) / 2; ++e) o[e] = pk(otherwise, otherwise);
    } else if (V >= 4 && vec) {
#pragma unroll
        for (int e = 0; e + 3 < V; e += 4) {
            const float4 q = c < width ? __ldg(reinterpret_cast<const float4*>(p + c + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
            o[e / 2] = pk(q.x, q.y);
            o[(e / 2 + 1) % ((V + 1) / 2)] = pk(q.z, q.w);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 2)
            o[e / 2] = pk(c + e < width ? __ldg(p + c + e) : 0.f, e + 1 < V && c + e + 1 < width ? __ldg(p + c + e + 1) : 0.f);
    }
}

// Threads that share a row of `vecs` vectors, a power of two: enough that a thread holds at most `most` vectors, more
// (down to one each) while the rows alone leave the SMs with less than about 1024 threads.
int row_lanes(int64_t rows, int vecs, int most, int least) {
    int lanes = least;
    while (lanes < kThreads && (int64_t)lanes * most < vecs) lanes *= 2;
    while (lanes < kThreads && lanes < vecs && rows * lanes < kSms * 1024) lanes *= 2;
    return lanes;
}

}  // namespace
}  // namespace ssd
