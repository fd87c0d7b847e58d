// k_group_norm_bf16.cu -- the grouped norm's kernels for bfloat16.
#include "group_norm.cuh"

namespace ssd {

int group_norm_forward_bf16(const GroupNormArgs& g, void* y, float* mean, float* rstd, cudaStream_t s) {
    return group_forward_type<__nv_bfloat16>(g, y, mean, rstd, s);
}
int group_norm_backward_bf16(const GroupNormArgs& g, const GroupNormGrads& d, float* partial, int* parts, cudaStream_t s) {
    return group_backward_type<__nv_bfloat16>(g, d, partial, parts, s);
}

}  // namespace ssd
