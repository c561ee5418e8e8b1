#include "delta_chain.cuh"

namespace dwp {

cudaError_t launch_delta_chain_back_bf16(const DeltaBackwardParams &p, const DeltaMaps &m, int pass, cudaStream_t s) {
    return chain_t<__nv_bfloat16, true>(p, m, pass, s);
}

}  // namespace dwp
