#include "delta_grad.cuh"

namespace dwp {

cudaError_t launch_delta_grad_f32(const DeltaBackwardParams &p, cudaStream_t s) { return grad_t<float>(p, s); }

}  // namespace dwp
