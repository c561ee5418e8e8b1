#include "delta_grad.cuh"

namespace dwp {

cudaError_t launch_delta_grad_f32(const DeltaBackwardParams &p, const DeltaMaps &m, cudaStream_t s) {
    return grad_t<float>(p, m, s);
}

}  // namespace dwp
