#include "delta_chain.cuh"

namespace dwp {

cudaError_t launch_delta_chain_back_f16(const DeltaBackwardParams &p, const DeltaMaps &m, int pass, cudaStream_t s) {
    return chain_t<__half, true>(p, m, pass, s);
}

}  // namespace dwp
