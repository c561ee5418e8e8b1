#include "delta_grad.cuh"

namespace dwp {

cudaError_t launch_delta_grad_f16(const DeltaBackwardParams &p, cudaStream_t s) { return grad_t<__half>(p, s); }

}  // namespace dwp
