#include "delta_grad.cuh"

namespace dwp {

cudaError_t launch_delta_grad_f16(const DeltaBackwardParams &p, const DeltaMaps &m, cudaStream_t s) {
    return grad_t<__half>(p, m, s);
}

}  // namespace dwp
