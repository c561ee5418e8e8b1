// The selective scan's walks over rows for bf16 activations.
#include "selscan_forward.cuh"

namespace dwp {

cudaError_t launch_selscan_bf16(const ScanParams &p, cudaStream_t s) { return scan_t<__nv_bfloat16>(p, s); }
cudaError_t launch_scan_walk_back_bf16(const ScanParams &p, cudaStream_t s) { return back_t<__nv_bfloat16>(p, s); }

}  // namespace dwp
