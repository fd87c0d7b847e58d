// k_selective_bwd_bf16.cu -- the selective scan's gradient on bfloat16 tensors.
#include "selective_backward.cuh"

namespace ssd {

int selective_backward_bf16(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s) {
    return backward_of<__nv_bfloat16>(a, g, ws, s);
}

}  // namespace ssd
