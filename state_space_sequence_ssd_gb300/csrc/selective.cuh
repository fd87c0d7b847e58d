// selective.cuh -- device helpers of the selective scan's kernels: the dt transform and the sum over the lanes that
// share a channel.
#pragma once

#include "ops.cuh"

namespace ssd {

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1].  log1p(e) / e is fitted on [0, 1] by a polynomial
// of degree 8 through the Chebyshev expansion (largest relative error 1.71e-7 with its float32 evaluation, over every e), so the
// result stays relatively exact where e is small, as a logarithm of 1 + e would not.  (Not in packed arithmetic: its
// constants would each take two moves, where a scalar instruction holds one.)
__device__ __forceinline__ float softplus(float v) {
    const float e = exp2_fast(-fabsf(v) * kLog2e);
    float p = 0.005253457929939032f;
    p = fmaf(p, e, -0.02958850748836994f);
    p = fmaf(p, e, 0.07836166769266129f);
    p = fmaf(p, e, -0.13674770295619965f);
    p = fmaf(p, e, 0.19111430644989014f);
    p = fmaf(p, e, -0.24844369292259216f);
    p = fmaf(p, e, 0.33319270610809326f);
    p = fmaf(p, e, -0.49999502301216125f);
    p = fmaf(p, e, 1.f);
    return fmaf(p, e, fmaxf(v, 0.f));
}

// v held to [lo, hi]; a NaN stays one (fminf and fmaxf would make it lo).
__device__ __forceinline__ float held_to(float v, float lo, float hi) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(lo));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(hi));
    return r;
}

// The effective dt of M values of raw dt with their bias added: softplus, limits.  The options are looked at once for
// all of them: a branch within each value's chain of dependent instructions would run the chains one after another.
// Without limits lo and hi are infinities; a step takes them without a branch, which would stand between its loads and their
// use (256 rows of 4096 x 16: 28.7 us, 31.2 with it), a prompt with one (2 x 4096 x 4096 x 16: 282 us, 285 without).
template <bool BRANCH, int M>
__device__ __forceinline__ void effective(float (&v)[M], const DtOpts& o) {
    if (o.softplus) {
#pragma unroll
        for (int i = 0; i < M; ++i) v[i] = softplus(v[i]);
    }
    if (!BRANCH || o.limit) {
#pragma unroll
        for (int i = 0; i < M; ++i) v[i] = held_to(v[i], o.lo, o.hi);
    }
}

// What arrives of s over tokens whose decays multiply to 2^v, and `own` that these tokens add.  The product may round to zero
// where none of its decays is: an infinite s stays infinite then, as it does token by token, and is no zero times infinity.
__device__ __forceinline__ float carried(float v, float s, float own) {
    return fabsf(s) == __int_as_float(0x7f800000) && v > -__int_as_float(0x7f800000) ? s + own : fmaf(exp2_fast(v), s, own);
}

// Sums R values over the lanes at offsets OFF, OFF / 2, ..., MIN.  While a lane holds several values it keeps one half
// and trades the other with its partner, so that R values cost about R shuffles.  The lane keeps the sums number
// which .. which + (values left) - 1, in v[0 ..].
template <int R, int OFF, int MIN>
__device__ __forceinline__ void fold_between(float* v, int lane, int& which) {
    if constexpr (OFF >= MIN) {
        if constexpr (R > 1) {
            constexpr int HALF = R / 2;
            const bool up = (lane & OFF) != 0;
#pragma unroll
            for (int j = 0; j < HALF; ++j) {
                const float mine = up ? v[j + HALF] : v[j];
                const float other = up ? v[j] : v[j + HALF];
                v[j] = mine + __shfl_xor_sync(0xffffffffu, other, OFF);
            }
            if (up) which += HALF;
            fold_between<HALF, OFF / 2, MIN>(v, lane, which);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], OFF);
            fold_between<1, OFF / 2, MIN>(v, lane, which);
        }
    }
}

// Lanes that share a channel, four state entries each: a power of two that covers dstate.
inline int selective_lanes(int dstate) {
    int lp = 2;
    while (lp * 4 < dstate) lp *= 2;
    return lp;
}

// Whether the token rows of x, dt, z (and of dense tensors of the same shape) are whole vectors of V channels, and
// those of B and C whole vectors of V entries.
inline bool rows_of(const SelectiveArgs& a, int V, const void* out1, const void* out2, size_t size) {
    return a.channels / a.ngroups % V == 0 && a.x_batch % V == 0 && a.x_token % V == 0 && a.dt_batch % V == 0 &&
           a.dt_token % V == 0 && (a.z == nullptr || (a.z_batch % V == 0 && a.z_token % V == 0)) &&
           aligned_to(a.x, V * size) && aligned_to(a.dt, V * size) && aligned_to(a.z, V * size) &&
           aligned_to(out1, V * size) && aligned_to(out2, V * size);
}
inline bool states_of(const SelectiveArgs& a, int V, size_t size) {
    return a.dstate % V == 0 && a.B_batch % V == 0 && a.B_token % V == 0 && a.C_batch % V == 0 && a.C_token % V == 0 &&
           aligned_to(a.B, V * size) && aligned_to(a.C, V * size);
}
inline bool rows_of_four(const SelectiveArgs& a, const void* out1, const void* out2, size_t size) {
    return rows_of(a, 4, out1, out2, size);
}
inline bool states_of_four(const SelectiveArgs& a, size_t size) { return states_of(a, 4, size); }

// How the forward pass runs: with wide lanes (four channels of eight entries) or narrow ones (two of four), the lanes
// that share a channel, threads of a block and its channels.
struct SelectiveShape {
    bool wide;
    int lp, threads, cc;
};
SelectiveShape selective_shape(const SelectiveArgs& a, bool wide);
int launch_selective_hop(const SelectiveArgs& a, int nchunks, float* hops, const float* dtsum, cudaStream_t s);
int selective_forward_bf16(const SelectiveArgs& a, const SelectivePlan& p, void* y, float* final_state, float* ws, cudaStream_t s);
int selective_forward_f16(const SelectiveArgs& a, const SelectivePlan& p, void* y, float* final_state, float* ws, cudaStream_t s);
int selective_forward_f32(const SelectiveArgs& a, const SelectivePlan& p, void* y, float* final_state, float* ws, cudaStream_t s);


// How the gradient runs: the tokens of a block, blocks of a row, blocks of a group's channels, and the floats of each part
// of its workspace.
struct SelectiveParts {
    int tokens, nblocks, tiles;  // of a block; blocks of a row; blocks of a group's channels
    size_t hops, nu0, dtsum, chan, dbc;  // floats of each part
    size_t total() const { return 2 * hops + nu0 + dtsum + chan + dbc; }
};
SelectiveParts selective_parts(const SelectiveArgs& a);
int selective_block_threads(const SelectiveArgs& a);
int launch_selective_hops(const SelectiveArgs& a, const SelectiveGrads& g, const SelectiveParts& p, float* hops, float* mus,
                          const float* nu0, const float* dtsum, cudaStream_t s);
int launch_selective_sums(const SelectiveArgs& a, const SelectiveGrads& g, const SelectiveParts& p, const float* dA_parts,
                          const float* chan, const float* dbc, cudaStream_t s);
int selective_backward_bf16(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s);
int selective_backward_f16(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s);
int selective_backward_f32(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s);

}  // namespace ssd
