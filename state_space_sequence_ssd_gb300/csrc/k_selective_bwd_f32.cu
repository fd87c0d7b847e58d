// k_selective_bwd_f32.cu -- the selective scan's gradient on float32 tensors.
#include "selective_backward.cuh"

namespace ssd {

int selective_backward_f32(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s) {
    return backward_of<float>(a, g, ws, s);
}

}  // namespace ssd
