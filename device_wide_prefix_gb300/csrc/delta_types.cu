// Gated delta rule: the chain's and the gradient's kernels by type (a
// translation unit each), the maps of their inputs, and the chain over
// sequences cut in parts.
#include <atomic>

#include "device.cuh"
#include "launch.h"

namespace dwp {

#ifdef DWP_DELTA_TEST
// Build for tests (-DDWP_DELTA_TEST=1): calls as where no tensor map can be made.
static std::atomic<int> delta_test_no_maps{0};
extern "C" void dwp_delta_test_no_maps(int on) { delta_test_no_maps = on; }
// And whose waits at one site run out (tensor.cuh, WaitSite; 0 for none).
static std::atomic<int> delta_test_site{0}, delta_test_skip{0};
extern "C" void dwp_delta_test_stall(int site, int skip) { delta_test_site = site, delta_test_skip = skip; }
void delta_stall(DeltaParams &p) { p.stall_site = delta_test_site, p.stall_skip = delta_test_skip; }
#endif

namespace {

using EncodeMap = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                               const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, by way of the runtime, so that nothing links the driver.
EncodeMap encode_map() {
#ifdef DWP_DELTA_TEST
    if (delta_test_no_maps) return nullptr;
#endif
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

// A map of rows [batch][rows][heads][size] for boxes `columns` wide, exchanged as
// tiles are if `tiles`.
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

cudaError_t chain_pass(dwp_dtype t, const DeltaBackwardParams &p, const DeltaMaps &m, bool back, int pass, cudaStream_t s) {
    if (back) {
        if (t == DWP_F32) return launch_delta_chain_back_f32(p, m, pass, s);
        return t == DWP_BF16 ? launch_delta_chain_back_bf16(p, m, pass, s) : launch_delta_chain_back_f16(p, m, pass, s);
    }
    if (t == DWP_F32) return launch_delta_chain_f32(p, m, pass, s);
    return t == DWP_BF16 ? launch_delta_chain_bf16(p, m, pass, s) : launch_delta_chain_f16(p, m, pass, s);
}

cudaError_t chain(dwp_dtype t, const DeltaBackwardParams &p, const DeltaMaps &m, bool back, cudaStream_t s) {
    if (p.f.parts == 1) return chain_pass(t, p, m, back, 0, s);
    cudaError_t err = chain_pass(t, p, m, back, 1, s);
    if (err == cudaSuccess) err = launch_delta_join(p.f, s);
    return err == cudaSuccess ? chain_pass(t, p, m, back, 2, s) : err;
}

constexpr int kJoinThreads = 256, kJoinCols = 16, kJoinKeys = 128, kJoinPitch = kJoinKeys + 1;
constexpr size_t kJoinBytes = sizeof(float) * (kJoinKeys * kJoinPitch + kJoinKeys * kJoinCols);

// start[part + 1] = map[part] start[part] + end[part], 16 columns a block.
__global__ void __launch_bounds__(kJoinThreads) delta_join_kernel(DeltaParams p) {
    extern __shared__ float sh[];
    float *map = sh, *S = sh + kJoinKeys * kJoinPitch;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, keys = p.keys, values = p.values, c0 = blockIdx.x * kJoinCols;
    const int k = tid / 2, c = tid % 2 * (kJoinCols / 2);
    for (int64_t part = 1; part + 1 < p.parts; ++part) {
        const int64_t at = (int64_t(blockIdx.z) * p.parts + part) * p.heads + blockIdx.y;
        const float *from = p.part_maps + at * keys * keys, *start = p.part_starts + at * keys * values;
        __syncthreads();
        for (int e = tid; e < keys * keys; e += kJoinThreads) map[e / keys * kJoinPitch + e % keys] = from[e];
        for (int e = tid; e < keys * kJoinCols; e += kJoinThreads) {
            const int col = c0 + e % kJoinCols;
            // the first start is pass 1's; the later ones this block wrote itself
            S[e] = col < values ? start[int64_t(e / kJoinCols) * values + col] : 0.0f;
        }
        __syncthreads();
        float s[kJoinCols / 2] = {};
        if (k < keys)
            for (int m = 0; m < keys; ++m) {
                const float x = map[k * kJoinPitch + m];
#pragma unroll
                for (int j = 0; j < kJoinCols / 2; ++j) s[j] = fmaf(x, S[m * kJoinCols + c + j], s[j]);
            }
        float *to = p.part_starts + (at + p.heads) * keys * values;
        const float *end = p.part_ends + at * keys * values;
#pragma unroll
        for (int j = 0; j < kJoinCols / 2; ++j)
            if (k < keys && c0 + c + j < values) {
                const int64_t e = int64_t(k) * values + c0 + c + j;
                to[e] = s[j] + end[e];
            }
        __threadfence_block();
    }
}

}  // namespace

DeltaMaps delta_maps(dwp_dtype t, const DeltaParams &p, const DeltaRows *grad_out) {
    DeltaMaps m = {};
    m.made = t == DWP_BF16 && p.wide && p.batch * p.rows > 0 &&
             delta_map(&m.k, p.k, p.batch, p.rows, p.key_heads, p.keys, 64, true) &&
             delta_map(&m.q, p.q, p.batch, p.rows, p.key_heads, p.keys, 64, true) &&
             delta_map(&m.v, grad_out ? *grad_out : p.v, p.batch, p.rows, p.heads, p.values, grad_out ? 64 : 128,
                       grad_out != nullptr);
    return m;
}

// Parts that a walk along a sequence is cut into: as many as fill the GPU's
// blocks in pass 1, eight chunks each at least, and three or none (of two parts
// the second would wait for the first as before).  Cut against uncut, bf16 heads
// of 128 x 128: 1 sequence x 8192 rows x 32 heads 466 us against 502, 32768 rows
// 1655 against 1961, the training step of 8192 rows x 16 heads 1044 against 1720.
// With more than 50 walks the two passes would be longer than the one; with
// offsets the parts would depend on what the host has not read.
int64_t delta_parts(int64_t walks, int64_t chunks) {
    if (walks < 1) return 1;
    int64_t parts = (kSMs / walks + 3) / 2;  // walks (2 parts - 3) blocks in pass 1
    if (parts > chunks / 8) parts = chunks / 8;
    return parts < 3 ? 1 : parts;
}

cudaError_t launch_delta_join(const DeltaParams &p, cudaStream_t s) {
    if (device_blocks(reinterpret_cast<const void *>(delta_join_kernel), kJoinThreads, kJoinBytes) == 0)
        return cudaErrorInvalidConfiguration;
    return launch_pdl(delta_join_kernel,
                      dim3(uint32_t((p.values + kJoinCols - 1) / kJoinCols), uint32_t(p.heads), uint32_t(p.sequences)),
                      dim3(kJoinThreads), kJoinBytes, s, p);
}

cudaError_t launch_delta_chain(dwp_dtype t, const DeltaParams &p, const DeltaMaps &m, cudaStream_t s) {
    DeltaBackwardParams b = {};
    b.f = p;
    return chain(t, b, m, false, s);
}
cudaError_t launch_delta_chain_back(dwp_dtype t, const DeltaBackwardParams &p, const DeltaMaps &m, cudaStream_t s) {
    return chain(t, p, m, true, s);
}

cudaError_t launch_delta_grad(dwp_dtype t, const DeltaBackwardParams &p, const DeltaMaps &m, cudaStream_t s) {
    if (t == DWP_F32) return launch_delta_grad_f32(p, m, s);
    return t == DWP_BF16 ? launch_delta_grad_bf16(p, m, s) : launch_delta_grad_f16(p, m, s);
}

}  // namespace dwp
