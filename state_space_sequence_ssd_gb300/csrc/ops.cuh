// ops.cuh -- what the layer operators (k_conv.cu, k_selective*.cu, k_norm.cu, k_gated.cu, k_group_norm*.cu, k_rotary.cu) share: the element types
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

// 2^v by the special function unit (relative error about 2^-22; results below 2^-126 are zero)
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / (1 + exp(-v)).  Past v = -88 the denominator overflows and its reciprocal is 0, the limit.
__device__ __forceinline__ float sigmoid(float v) { return rcp_fast(1.f + exp2_fast(v * -kLog2e)); }

// Two float32 values in one register pair, for sm_100's packed arithmetic (one instruction, each lane rounded as
// a separate instruction would be; the multiplier takes as long as for two, the issue slot is saved).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pk(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpk(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ float sum2(f32x2 v) {
    float lo, hi;
    unpk(v, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 exp2_2(f32x2 v) {
    float lo, hi;
    unpk(v, lo, hi);
    return pk(exp2_fast(lo), exp2_fast(hi));
}
__device__ __forceinline__ f32x2 sigmoid2(f32x2 v) {  // constants: one in a scalar instruction, two moves in a packed one
    float lo, hi;
    unpk(v, lo, hi);
    return pk(sigmoid(lo), sigmoid(hi));
}

// V consecutive elements as they lie in memory.  They stay packed words until get() unpacks one: a load whose halves
// are taken apart at once would be waited for at once.
template <typename T, int V>
struct Vec {
    static constexpr int BYTES = sizeof(T) * V, WORDS = (BYTES + 3) / 4;
    static_assert(BYTES == 2 || BYTES == 4 || BYTES == 8 || BYTES == 16, "one access");
    uint32_t w[WORDS];

    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
        else return __half2float(__ushort_as_half((unsigned short)((i & 1) ? (w[i / 2] >> 16) : (w[i / 2] & 0xffffu))));
    }
    // each value rounded once
    __device__ __forceinline__ static Vec of(const float (&v)[V]) {
        Vec r;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const float hi = 2 * i + 1 < V ? v[2 * i + 1 < V ? 2 * i + 1 : 0] : 0.f;
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], hi);
                    r.w[i] = *reinterpret_cast<const uint32_t*>(&p);
                } else {
                    const __half2 p = __floats2half2_rn(v[2 * i], hi);
                    r.w[i] = *reinterpret_cast<const uint32_t*>(&p);
                }
            }
        }
        return r;
    }
    // elements 2 i and 2 i + 1
    __device__ __forceinline__ f32x2 pair(int i) const;
    __device__ __forceinline__ static Vec of_pairs(const f32x2 (&v)[(V + 1) / 2]);
    __device__ __forceinline__ static Vec zero() {
        Vec r;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r.w[i] = 0u;
        return r;
    }
};

// The bits of one element.
template <typename T>
__device__ __forceinline__ uint32_t bits_at(const T* p) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const uint32_t*>(p);
    else return *reinterpret_cast<const unsigned short*>(p);
}

// V elements at p, those from `valid` on taken as zero.  `vec`: p is aligned to the whole vector and either all of
// its elements are valid or none.  KEEP: the memory may be written by this kernel (else the read-only path).
template <typename T, int V, bool KEEP = false>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p, int valid, bool vec) {
    using R = Vec<T, V>;
    R r = R::zero();
    if (vec) {
        if (valid > 0) {
            if constexpr (R::BYTES == 16) {
                const uint4 q = KEEP ? *reinterpret_cast<const uint4*>(p) : __ldg(reinterpret_cast<const uint4*>(p));
                r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
            } else if constexpr (R::BYTES == 8) {
                const uint2 q = KEEP ? *reinterpret_cast<const uint2*>(p) : __ldg(reinterpret_cast<const uint2*>(p));
                r.w[0] = q.x; r.w[1] = q.y;
            } else if constexpr (R::BYTES == 4) {
                r.w[0] = KEEP ? *reinterpret_cast<const uint32_t*>(p) : __ldg(reinterpret_cast<const uint32_t*>(p));
            } else {
                r.w[0] = KEEP ? *reinterpret_cast<const unsigned short*>(p) : __ldg(reinterpret_cast<const unsigned short*>(p));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) r.w[sizeof(T) == 4 ? i : i / 2] |= bits_at(p + i) << ((sizeof(T) == 2 && (i & 1)) ? 16 : 0);
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& r, int valid, bool vec) {
    using R = Vec<T, V>;
    if (vec) {
        if (valid <= 0) return;
        if constexpr (R::BYTES == 16) *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        else if constexpr (R::BYTES == 8) *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
        else if constexpr (R::BYTES == 4) *reinterpret_cast<uint32_t*>(p) = r.w[0];
        else *reinterpret_cast<unsigned short*>(p) = (unsigned short)r.w[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) {
                if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(p + i) = r.w[i];
                else *reinterpret_cast<unsigned short*>(p + i) = (unsigned short)((i & 1) ? r.w[i / 2] >> 16 : r.w[i / 2] & 0xffffu);
            }
    }
}

template <typename T, int V>
__device__ __forceinline__ f32x2 Vec<T, V>::pair(int i) const {
    if constexpr (V == 1) return pk(get(0), 0.f);
    else if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        return pk(f.x, f.y);
    } else return pk(get(2 * i), get(2 * i + 1));
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> Vec<T, V>::of_pairs(const f32x2 (&v)[(V + 1) / 2]) {
    float f[V + 1];
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) unpk(v[i], f[2 * i], f[2 * i + 1]);
    float g[V];
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = f[i];
    return of(g);
}

// Sixteen bytes from global to shared memory without a register between; zeros where `live` is false.
__device__ __forceinline__ void copy16(void* to, const void* from, bool live) {
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
    const int bytes = live ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(bytes) : "memory");
}
// Four bytes from global to shared memory without a register between.
__device__ __forceinline__ void copy4(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

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

// Blocks of a grid in y and in z; SMs that the launch rules mean to fill.
constexpr int kMaxGrid = 65535, kSms = 152;

inline bool aligned_to(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Kernel kinds of the layer operators, after those of the scan.
enum LayerKind {
    kKindConv = kNumKinds,
    kKindConvBwd,
    kKindConvStep,
    kKindSelective,
    kKindSelectiveBwd,
    kKindSelectiveStep,
    kKindNorm,
    kKindNormBwd,
    kKindGated,
    kKindGatedBwd,
    kKindGatedStep,
    kKindGroupNorm,
    kKindGroupNormBwd,
    kKindRotary,
    kAllKinds
};

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
// How the forward pass runs: the width of its lanes, the chunks that the sequence is split into (1: no split); and the
// workspace in bytes that this takes.
struct SelectivePlan {
    bool wide;
    int chunks;
};
SelectivePlan selective_plan(const SelectiveArgs& a, int sms);
size_t selective_workspace(const SelectiveArgs& a, const SelectivePlan& p);
int launch_selective_forward(const SelectiveArgs& a, const SelectivePlan& p, void* y, float* final_state, float* ws,
                             cudaStream_t s);

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
// partial: layer_norm_parts(rows, sms) x 2 x width float32
int layer_norm_parts(int64_t rows, int sms);
int launch_layer_norm_backward(int dtype, const void* x, int64_t x_row, const float* weight, const float* mean,
                               const float* rstd, const void* dy, int64_t dy_row, int64_t rows, int width, void* dx,
                               float* dweight, float* dbias, float* partial, int parts, cudaStream_t s);

struct GatedArgs {
    int dtype, batch, seqlen, channels;
    const void *x, *r, *i;
    int64_t x_batch, x_token, r_batch, r_token, i_batch, i_token;
    const float* A;     // (channels)
    const float* init;  // (batch, channels) or nullptr
    const int* lengths;
};
struct GatedGrads {
    const void* dy;       // dense
    const float* dfinal;  // or nullptr
    void *dx, *dr, *di;
    float *dA, *dinit;  // dinit may be nullptr
};
// Floats of the states that the forward pass keeps for the gradient, and of the gradient's sums of parts.
size_t gated_states_floats(const GatedArgs& g);
size_t gated_sums_floats(const GatedArgs& g);
int launch_gated_forward(const GatedArgs& g, void* y, float* final_state, float* states, cudaStream_t s);
int launch_gated_backward(const GatedArgs& g, const GatedGrads& d, const float* states, float* partial, cudaStream_t s);
int launch_gated_step(const GatedArgs& g, float* state, const int* slots, int nslots, void* y, int* err, cudaStream_t s);

// The column sums of a norm's gradient: dweight and dbias (either may be nullptr) from `parts` rows of 2 x width, whose
// second halves are not read without a dbias.
int launch_norm_sums(int kind, const float* partial, int parts, int width, float* dweight, float* dbias, cudaStream_t s);

enum Gate { kGateNone = SSD_GATE_NONE, kGateSilu = SSD_GATE_SILU, kGateAfter = SSD_GATE_AFTER, kGateBefore = SSD_GATE_BEFORE };
struct GroupNormArgs {
    int dtype;
    int64_t rows;
    int width, groups, gate;
    bool rms;
    float eps;
    const void *x, *z;  // z with kGateAfter and kGateBefore only
    int64_t x_row, z_row;
    const float *weight, *bias;  // (width) or nullptr
};
struct GroupNormGrads {
    const float *mean, *rstd;  // (rows, groups); mean is nullptr where rms
    const void* dy;
    int64_t dy_row;
    void *dx, *dz;
    bool want_dbias;
};
int group_norm_forward_bf16(const GroupNormArgs& g, void* y, float* mean, float* rstd, cudaStream_t s);
int group_norm_forward_f16(const GroupNormArgs& g, void* y, float* mean, float* rstd, cudaStream_t s);
int group_norm_forward_f32(const GroupNormArgs& g, void* y, float* mean, float* rstd, cudaStream_t s);
// partial: *parts x 2 x width float32, or nullptr where no column sums are wanted; *parts becomes the number of them that are written
int group_norm_backward_bf16(const GroupNormArgs& g, const GroupNormGrads& d, float* partial, int* parts, cudaStream_t s);
int group_norm_backward_f16(const GroupNormArgs& g, const GroupNormGrads& d, float* partial, int* parts, cudaStream_t s);
int group_norm_backward_f32(const GroupNormArgs& g, const GroupNormGrads& d, float* partial, int* parts, cudaStream_t s);

struct RotaryArgs {
    int dtype, batch, seqlen, dim, turned;
    bool interleaved, inverse;
    float scale;
    int heads[2];  // the second may be 0
    const void* in[2];
    int64_t batch_stride[2], token_stride[2];
    void* out[2];  // dense
    const unsigned long long* table;  // (turned / 2)
    const int* positions;             // (batch), (batch, seqlen) where `each`, or nullptr
    bool each;
    const int* lengths;
};
int launch_rotary(const RotaryArgs& g, cudaStream_t s);

// Workspace, error words and device size, implemented in ssd_api.cu.
int take_workspace(void** ptr, size_t bytes, cudaStream_t s);
int* error_words();
Ctl wait_control(int kind);  // of a kernel of this kind: its error words, wait limit and test hook
int multiprocessors();

}  // namespace ssd
