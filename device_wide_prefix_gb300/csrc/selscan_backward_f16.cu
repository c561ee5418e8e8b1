// The selective scan's gradient for f16 activations.
#include "selscan_backward.cuh"

namespace dwp {

cudaError_t launch_selscan_backward_f16(const ScanBackwardParams &q, cudaStream_t s) { return backward_t<__half>(q, s); }

}  // namespace dwp
