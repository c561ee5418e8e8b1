// Gated delta rule: the chain's and the gradient's kernels by type (a
// translation unit each).
#include "launch.h"

namespace dwp {

namespace {

cudaError_t chain(dwp_dtype t, const DeltaBackwardParams &p, bool back, cudaStream_t s) {
    if (t == DWP_F32) return launch_delta_chain_f32(p, back, s);
    return t == DWP_BF16 ? launch_delta_chain_bf16(p, back, s) : launch_delta_chain_f16(p, back, s);
}

}  // namespace

cudaError_t launch_delta_chain(dwp_dtype t, const DeltaParams &p, cudaStream_t s) {
    DeltaBackwardParams b = {};
    b.f = p;
    return chain(t, b, false, s);
}
cudaError_t launch_delta_chain_back(dwp_dtype t, const DeltaBackwardParams &p, cudaStream_t s) {
    return chain(t, p, true, s);
}

cudaError_t launch_delta_grad(dwp_dtype t, const DeltaBackwardParams &p, cudaStream_t s) {
    if (t == DWP_F32) return launch_delta_grad_f32(p, s);
    return t == DWP_BF16 ? launch_delta_grad_bf16(p, s) : launch_delta_grad_f16(p, s);
}

}  // namespace dwp
