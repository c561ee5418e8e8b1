// The selective scan's forward for bf16 activations.
#include "selscan_forward.cuh"

namespace dwp {

cudaError_t launch_selscan_bf16(const ScanParams &p, cudaStream_t s) { return scan_t<__nv_bfloat16>(p, s); }

}  // namespace dwp
