#include "delta_chain.cuh"

namespace dwp {

cudaError_t launch_delta_chain_f16(const DeltaBackwardParams &p, bool back, cudaStream_t s) {
    return back ? chain_t<__half, true>(p, s) : chain_t<__half, false>(p, s);
}

}  // namespace dwp
