#include "delta_chain.cuh"

namespace dwp {

cudaError_t launch_delta_chain_bf16(const DeltaBackwardParams &p, int pass, cudaStream_t s) {
    return chain_t<__nv_bfloat16, false>(p, pass, s);
}

}  // namespace dwp
