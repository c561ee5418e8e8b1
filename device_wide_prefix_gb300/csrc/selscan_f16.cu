// The selective scan's forward for f16 activations.
#include "selscan_forward.cuh"

namespace dwp {

cudaError_t launch_selscan_f16(const ScanParams &p, cudaStream_t s) { return scan_t<__half>(p, s); }

}  // namespace dwp
