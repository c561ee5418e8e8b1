#include "delta_chain.cuh"

namespace dwp {

cudaError_t launch_delta_chain_bf16(const DeltaBackwardParams &p, bool back, cudaStream_t s) {
    return back ? chain_t<__nv_bfloat16, true>(p, s) : chain_t<__nv_bfloat16, false>(p, s);
}

}  // namespace dwp
