// The selective scan's walks over rows for f16 activations.
#include "selscan_forward.cuh"

namespace dwp {

cudaError_t launch_selscan_f16(const ScanParams &p, cudaStream_t s) { return scan_t<__half>(p, s); }
cudaError_t launch_scan_walk_back_f16(const ScanParams &p, cudaStream_t s) { return back_t<__half>(p, s); }

}  // namespace dwp
