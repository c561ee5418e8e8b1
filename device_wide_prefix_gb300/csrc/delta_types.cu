// Gated delta rule: the chain's and the gradient's kernels by type (a
// translation unit each), and the maps of their inputs.
#include <atomic>

#include "launch.h"

namespace dwp {

namespace {

using EncodeMap = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                               const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, by way of the runtime, so that nothing links the driver.
EncodeMap encode_map() {
    static std::atomic<void *> known{nullptr};
    void *f = known.load();
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        known.store(f);
    }
    return reinterpret_cast<EncodeMap>(f);
}

}  // namespace

bool delta_map(CUtensorMap *map, const DeltaRows &r, int64_t batch, int64_t rows, int64_t heads, int64_t size, int columns,
               bool tiles) {
    const EncodeMap encode = encode_map();
    if (!encode) return false;
    const cuuint64_t dims[4] = {cuuint64_t(size), cuuint64_t(heads), cuuint64_t(rows), cuuint64_t(batch)};
    // the stride of a single head, row or entry is not used, and may be anything
    const cuuint64_t strides[3] = {cuuint64_t(heads > 1 ? r.head : size) * 2, cuuint64_t(rows > 1 ? r.row : size) * 2,
                                   cuuint64_t(batch > 1 ? r.batch : size) * 2};
    for (cuuint64_t s : strides)
        if (s >= (cuuint64_t(1) << 40)) return false;
    const cuuint32_t box[4] = {cuuint32_t(columns), 1, 64, 1}, step[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, r.data, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  tiles ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

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
