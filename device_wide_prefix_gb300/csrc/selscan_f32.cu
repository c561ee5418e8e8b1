// The selective scan's walks over rows for f32 activations.
#include "selscan_forward.cuh"

namespace dwp {

cudaError_t launch_selscan_f32(const ScanParams &p, cudaStream_t s) { return scan_t<float>(p, s); }
cudaError_t launch_scan_walk_back_f32(const ScanParams &p, cudaStream_t s) { return back_t<float>(p, s); }

}  // namespace dwp
