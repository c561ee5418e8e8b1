#include "delta_chain.cuh"

namespace dwp {

cudaError_t launch_delta_chain_f32(const DeltaBackwardParams &p, int pass, cudaStream_t s) {
    return chain_t<float, false>(p, pass, s);
}

}  // namespace dwp
