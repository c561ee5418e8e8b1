// The selective scan's gradient for f32 activations.
#include "selscan_backward.cuh"

namespace dwp {

cudaError_t launch_selscan_backward_f32(const ScanBackwardParams &q, cudaStream_t s) { return backward_t<float>(q, s); }

}  // namespace dwp
