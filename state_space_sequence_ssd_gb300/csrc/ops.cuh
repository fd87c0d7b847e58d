// ops.cuh -- what the layer operators (k_conv.cu, k_selective*.cu, k_norm.cu) share: the element types
// of their tensors, vector loads that fall back to single elements, and the launchers' declarations.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace ssd {

// ------------------------------------------------------------------ element types (ssd_dtype)
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }

// rounded once, to nearest even
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// V consecutive elements as one access of V * sizeof(T) bytes (at most 16)
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// V elements at p, those from `valid` on taken as zero.  `vec`: p is aligned to the whole vector.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p, int valid, bool vec) {
    Vec<T, V> r;
    if (vec && valid >= V) {
        r = *reinterpret_cast<const Vec<T, V>*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r.e[i] = i < valid ? p[i] : from_f32<T>(0.f);
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& r, int valid, bool vec) {
    if (vec && valid >= V) {
        *reinterpret_cast<Vec<T, V>*>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) p[i] = r.e[i];
    }
}

// 1 / (1 + exp(-v)).  Past v = -88 the denominator is beyond 2^126 and the approximate quotient 0, the limit.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// A row's length, held to [0, seqlen] (no lengths: the whole row).
__device__ __forceinline__ int row_length(const int* lengths, int b, int seqlen) {
    return lengths == nullptr ? seqlen : min(max(lengths[b], 0), seqlen);
}

// The pool slot of row b, or -1 where the row is idle.  A slot past the pool is idle too, and raises the
// slot flag of the device error words.
__device__ __forceinline__ int row_slot(const int* slots, int b, int nslots, int* err) {
    if (slots == nullptr) return b;
    const int s = slots[b];
    if (s >= nslots) {
        if (err != nullptr) atomicOr(err + 2, 1);
        return -1;
    }
    return s;
}

// ------------------------------------------------------------------ launchers (arguments are checked by ops_api.cu)

// Up to three dense row-major output (or gradient) pieces side by side: piece i holds n[i] channels.
struct Pieces {
    void* p[3] = {nullptr, nullptr, nullptr};
    int n[3] = {0, 0, 0};
    int f32[3] = {0, 0, 0};  // gradients: the piece is float32 whatever the operator's type
};

struct ConvArgs {
    int dtype, batch, seqlen, channels, width, silu;
    const void* x;
    int64_t x_batch, x_token;  // strides of x in elements
    const float* weight;       // (channels, width)
    const float* bias;         // (channels) or nullptr
    const void* init;          // (batch, width - 1, channels) or nullptr
    const int* lengths;        // (batch) or nullptr
};
int launch_conv_forward(const ConvArgs& a, const Pieces& y, void* final_state, cudaStream_t s);
// partial: conv_backward_rows(a) x channels x (width + 1) float32, the row sums of dweight and dbias
int conv_backward_rows(const ConvArgs& a);
int launch_conv_backward(const ConvArgs& a, const Pieces& dy, const void* dfinal, void* dx, int64_t dx_batch,
                         int64_t dx_token, float* dweight, float* dbias, void* dinit, float* partial, cudaStream_t s);
int launch_conv_step(const ConvArgs& a, void* state, const int* slots, int nslots, const Pieces& y, int* err,
                     cudaStream_t s);

struct SelectiveArgs {
    int dtype, batch, seqlen, channels, ngroups, dstate;
    const void *x, *dt, *B, *C, *z;  // z may be nullptr
    int64_t x_batch, x_token, dt_batch, dt_token, B_batch, B_token, C_batch, C_token, z_batch, z_token;
    const float* A;     // (channels, dstate)
    const float* D;     // (channels) or nullptr
    const float* init;  // (batch, channels, dstate) or nullptr
    const int* lengths;
    DtOpts dto;
};
// Chunks that the forward pass splits the sequence into (1: no split), and the float32 workspace it needs.
int selective_chunks(const SelectiveArgs& a, int sms);
size_t selective_workspace(const SelectiveArgs& a, int chunks);
int launch_selective_forward(const SelectiveArgs& a, int chunks, void* y, float* final_state, float* ws, cudaStream_t s);

struct SelectiveGrads {
    const void* dy;       // dense
    const float* dfinal;  // or nullptr
    void *dx, *ddt, *dz;  // dz with z only
    float *dA, *dB, *dC, *dD, *ddt_bias, *dinit;  // dD, ddt_bias, dinit may be nullptr
};
size_t selective_backward_workspace(const SelectiveArgs& a);
int launch_selective_backward(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s);
int launch_selective_step(const SelectiveArgs& a, float* state, const int* slots, int nslots, void* y, int* err,
                          cudaStream_t s);

int launch_layer_norm_forward(int dtype, const void* x, int64_t x_row, const float* weight, const float* bias, float eps,
                              int64_t rows, int width, void* y, float* mean, float* rstd, cudaStream_t s);
// partial: layer_norm_parts(rows, width, sms) x 2 x width float32
int layer_norm_parts(int64_t rows, int width, int sms);
int launch_layer_norm_backward(int dtype, const void* x, int64_t x_row, const float* weight, const float* mean,
                               const float* rstd, const void* dy, int64_t dy_row, int64_t rows, int width, void* dx,
                               float* dweight, float* dbias, float* partial, int parts, cudaStream_t s);

// Workspace, error words and device size, implemented in ssd_api.cu.
int take_workspace(void** ptr, size_t bytes, cudaStream_t s);
int* error_words();
int multiprocessors();

}  // namespace ssd
