// k_group_norm_f32.cu -- the grouped norm's kernels for float32.
#include "group_norm.cuh"

namespace ssd {

int group_norm_forward_f32(const GroupNormArgs& g, void* y, float* mean, float* rstd, cudaStream_t s) {
    return group_forward_type<float>(g, y, mean, rstd, s);
}
int group_norm_backward_f32(const GroupNormArgs& g, const GroupNormGrads& d, float* partial, int* parts, cudaStream_t s) {
    return group_backward_type<float>(g, d, partial, parts, s);
}

}  // namespace ssd
