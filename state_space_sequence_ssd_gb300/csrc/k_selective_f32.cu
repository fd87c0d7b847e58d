// k_selective_f32.cu -- the selective scan's forward pass on float32 tensors.
#include "selective_forward.cuh"

namespace ssd {

int selective_forward_f32(const SelectiveArgs& a, const SelectivePlan& p, void* y, float* final_state, float* ws,
                          cudaStream_t s) {
    return forward_of<float>(a, p, y, final_state, ws, s);
}

}  // namespace ssd
