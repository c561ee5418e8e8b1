// Selective state space scan: what its forward passes share whatever the
// type, and the choice of the type.
#include "selscan.cuh"

namespace dwp {

namespace {

// Carries the states over the chunks of a batch entry, in place: entry k
// becomes the state after chunk k.
__global__ void __launch_bounds__(256) carry_kernel(ScanParams p) {
    pdl_trigger();
    pdl_wait();
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x, per = p.channels * p.states;
    if (i >= per) return;
    const int64_t c = i / p.states;
    const float A2 = 0.5f * decay_rate(p.A[i]);
    const int64_t first = int64_t(blockIdx.y) * (p.chunks - 1);
    float *st = p.carry + first * per + i;
    const float *sum = p.carry_sum + first * p.channels + c;
    const uint32_t *head = p.carry_head + first;
    const int64_t entries = p.chunks - 1;
    constexpr int kBatch = 16;  // loads in flight: the stores between them would hold the later ones back
    float h = 0.0f;
    for (int64_t k0 = 0; k0 < entries; k0 += kBatch) {
        float e[kBatch], d[kBatch];
        bool cut[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t k = min(k0 + i, entries - 1);
            e[i] = st[k * per], d[i] = sum[k * p.channels], cut[i] = head[k] != 0u;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            // a chunk with a head takes nothing from before it, and from a zero
            // state nothing comes even where the product of decays overflows
            // the exponential of half the sum, twice: the product of a chunk's
            // decays may be past f32's range where the state times it is not
            const float a = ex2(A2 * d[i]);
            h = cut[i] || h == 0.0f ? e[i] : fmaf(h * a, a, e[i]);
            if (k0 + i < entries) st[(k0 + i) * per] = h;
        }
    }
}

// One code word per packed row: its segment, and whether it is the segment's
// first or last row.
__global__ void __launch_bounds__(256)
    segment_map_kernel(const uint32_t *offsets, uint32_t nseg, uint32_t rows, uint32_t *map) {
    pdl_trigger();
    pdl_wait();
    const uint32_t t = blockIdx.x * 256u + threadIdx.x;
    if (t >= rows) return;
    const uint32_t s = segment_of(offsets, nseg, t);
    uint32_t code = kRowOutside;
    if (s < nseg && offsets[s] <= t)
        code = s | (offsets[s] == t ? kRowHead : 0u) | (min(offsets[s + 1], rows) == t + 1u ? kRowTail : 0u);
    map[t] = code;
}

}  // namespace

cudaError_t launch_carry(const ScanParams &p, cudaStream_t s) {
    return launch_pdl(carry_kernel, dim3(uint32_t((p.channels * p.states + 255) / 256), uint32_t(p.batch)), dim3(256), 0,
                      s, p);
}

cudaError_t launch_segment_map(const uint32_t *offsets, uint32_t nseg, uint32_t rows, uint32_t *map,
                               cudaStream_t s) {
    return launch_pdl(segment_map_kernel, dim3((rows + 255u) / 256u), dim3(256), 0, s, offsets, nseg, rows, map);
}

int64_t scan_warp_channels(int64_t states) {
    return states <= 16 ? 64 : states <= 32 ? 32 : states <= 64 ? 16 : 8;
}

int64_t scan_block_channels(int64_t states) {
    return states <= 16 ? 32 : states <= 32 ? 16 : states <= 64 ? 8 : 4;
}

cudaError_t launch_scan_walk_back(dwp_dtype t, const ScanParams &p, cudaStream_t s) {
    if (t == DWP_F32) return launch_scan_walk_back_f32(p, s);
    if (t == DWP_BF16) return launch_scan_walk_back_bf16(p, s);
    return launch_scan_walk_back_f16(p, s);
}

cudaError_t launch_selscan_backward(dwp_dtype t, const ScanBackwardParams &q, cudaStream_t s) {
    if (t == DWP_F32) return launch_selscan_backward_f32(q, s);
    if (t == DWP_BF16) return launch_selscan_backward_bf16(q, s);
    return launch_selscan_backward_f16(q, s);
}

cudaError_t launch_selscan(dwp_dtype t, const ScanParams &p, cudaStream_t s) {
    if (t == DWP_F32) return launch_selscan_f32(p, s);
    if (t == DWP_BF16) return launch_selscan_bf16(p, s);
    return launch_selscan_f16(p, s);
}

}  // namespace dwp
