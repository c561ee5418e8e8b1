#include "delta_chain.cuh"

namespace dwp {

cudaError_t launch_delta_chain_f16(const DeltaBackwardParams &p, const DeltaMaps &m, int pass, cudaStream_t s) {
    return chain_t<__half, false>(p, m, pass, s);
}

}  // namespace dwp
