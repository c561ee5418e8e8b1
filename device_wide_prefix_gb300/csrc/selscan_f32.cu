// The selective scan's forward for f32 activations.
#include "selscan_forward.cuh"

namespace dwp {

cudaError_t launch_selscan_f32(const ScanParams &p, cudaStream_t s) { return scan_t<float>(p, s); }

}  // namespace dwp
