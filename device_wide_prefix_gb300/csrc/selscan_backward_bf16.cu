// The selective scan's gradient for bf16 activations.
#include "selscan_backward.cuh"

namespace dwp {

cudaError_t launch_selscan_backward_bf16(const ScanBackwardParams &q, cudaStream_t s) { return backward_t<__nv_bfloat16>(q, s); }

}  // namespace dwp
