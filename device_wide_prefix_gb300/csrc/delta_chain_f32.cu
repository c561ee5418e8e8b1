#include "delta_chain.cuh"

namespace dwp {

cudaError_t launch_delta_chain_f32(const DeltaBackwardParams &p, bool back, cudaStream_t s) {
    return back ? chain_t<float, true>(p, s) : chain_t<float, false>(p, s);
}

}  // namespace dwp
