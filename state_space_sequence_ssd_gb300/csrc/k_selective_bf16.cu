// k_selective_bf16.cu -- the selective scan's forward pass on bfloat16 tensors.
#include "selective_forward.cuh"

namespace ssd {

int selective_forward_bf16(const SelectiveArgs& a, const SelectivePlan& p, void* y, float* final_state, float* ws,
                          cudaStream_t s) {
    return forward_of<__nv_bfloat16>(a, p, y, final_state, ws, s);
}

}  // namespace ssd
