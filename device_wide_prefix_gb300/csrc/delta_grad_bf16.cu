#include "delta_grad.cuh"

namespace dwp {

cudaError_t launch_delta_grad_bf16(const DeltaBackwardParams &p, const DeltaMaps &m, cudaStream_t s) {
    return grad_t<__nv_bfloat16>(p, m, s);
}

}  // namespace dwp
