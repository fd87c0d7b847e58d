// selective.cuh -- device helpers of the selective scan's kernels: the dt transform and the sum over the lanes that
// share a channel.
#pragma once

#include "ops.cuh"

namespace ssd {

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1].  log1p(e) / e is fitted on [0, 1] by a polynomial
// of degree 8 through the Chebyshev expansion (largest relative error 1.5e-7 with its float32 evaluation), so the
// result stays relatively exact where e is small, as a logarithm of 1 + e would not.
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

// The effective dt of one channel: bias (already looked up), softplus, limits.
__device__ __forceinline__ float effective(float v, float bias, const DtOpts& o) {
    v += bias;
    if (o.softplus) v = softplus(v);
    if (o.limit) v = fminf(fmaxf(v, o.lo), o.hi);
    return v;
}

// Sums R values each over the lanes of a group (lane offsets OFF, OFF / 2, ..., 1): while a lane holds several
// values it keeps one half and trades the other with its partner.  The lane ends up with the full sum of one value,
// whose index is added to `which`.
template <int R, int OFF>
__device__ __forceinline__ float fold_lanes(const float (&v)[R], int lane, int& which) {
    if constexpr (R == 1) {
        float t = v[0];
#pragma unroll
        for (int o = OFF; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        return t;
    } else {
        constexpr int HALF = R / 2;
        const bool up = (lane & OFF) != 0;
        float w[HALF];
#pragma unroll
        for (int j = 0; j < HALF; ++j) {
            const float mine = up ? v[j + HALF] : v[j];
            const float other = up ? v[j] : v[j + HALF];
            w[j] = mine + __shfl_xor_sync(0xffffffffu, other, OFF);
        }
        if (up) which += HALF;
        return fold_lanes<HALF, OFF / 2>(w, lane, which);
    }
}

// Lanes that share a channel, four state entries each: a power of two that covers dstate.
inline int selective_lanes(int dstate) {
    int lp = 2;
    while (lp * 4 < dstate) lp *= 2;
    return lp;
}

inline bool aligned_to(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Whether the token rows of x, dt, z (and a dense output) can be read in vectors of four channels, and B and C in
// vectors of four entries.
inline bool rows_of_four(const SelectiveArgs& a, const void* out1, const void* out2, size_t size) {
    return a.channels / a.ngroups % 4 == 0 && a.x_batch % 4 == 0 && a.x_token % 4 == 0 && a.dt_batch % 4 == 0 &&
           a.dt_token % 4 == 0 && (a.z == nullptr || (a.z_batch % 4 == 0 && a.z_token % 4 == 0)) &&
           aligned_to(a.x, 4 * size) && aligned_to(a.dt, 4 * size) && aligned_to(a.z, 4 * size) &&
           aligned_to(out1, 4 * size) && aligned_to(out2, 4 * size);
}
inline bool states_of_four(const SelectiveArgs& a, size_t size) {
    return a.dstate % 4 == 0 && a.B_batch % 4 == 0 && a.B_token % 4 == 0 && a.C_batch % 4 == 0 && a.C_token % 4 == 0 &&
           aligned_to(a.B, 4 * size) && aligned_to(a.C, 4 * size);
}

}  // namespace ssd
