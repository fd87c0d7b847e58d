// k_selective_bwd_f16.cu -- the selective scan's gradient on float16 tensors.
#include "selective_backward.cuh"

namespace ssd {

int selective_backward_f16(const SelectiveArgs& a, const SelectiveGrads& g, float* ws, cudaStream_t s) {
    return backward_of<__half>(a, g, ws, s);
}

}  // namespace ssd
