// Host-side launch helpers and the kernel launchers behind the C entry points.
#pragma once

#include <cuda_runtime.h>

#include "common.h"

namespace dwp {

// Launch `kernel` with programmatic stream serialisation: it may begin while
// the previous kernel on `stream` finishes, and waits for it (pdl_wait)
// before it touches global memory.  Hides most of one launch latency per
// kernel boundary.
template <class... KArgs, class... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Zero [a, a + a_bytes) and [b, b + b_bytes) with one kernel on `stream`
// (launched like every other kernel here, so the kernel after it can start
// early).  Both pointers 4-byte aligned and both sizes multiples of 4 bytes;
// a null pointer or a zero size skips that range.
cudaError_t launch_clear(void *a, size_t a_bytes, void *b, size_t b_bytes, cudaStream_t stream);

// Resident blocks of `kernel` on the current device (SM count x blocks per
// SM at this block size and dynamic shared memory).  Also raises the
// kernel's dynamic shared-memory limit to `smem_bytes`.  Cached per device
// and kernel.  Returns 0 if the kernel cannot be resident at all.
int device_blocks(const void *kernel, int threads, size_t smem_bytes);

// Inputs of at most this many elements take the small-input plain scan
// (scan_small.cu: one block per tile); larger ones the persistent pipelined
// kernel (scan.cu).  Measured on GB300: at 2^23 the small-input kernel takes
// 19.3 us and the pipelined one 22.8; at 2^24, 43.3 against 34.4.
#ifndef DWP_SCAN_SMALL_LOG2
#define DWP_SCAN_SMALL_LOG2 23
#endif
constexpr uint64_t kScanSmallMax = uint64_t(1) << DWP_SCAN_SMALL_LOG2;
// Elements per tile of the large-input plain scan kernel.
uint32_t scan_tile_elems();
// Descriptors the small-input kernel needs for n <= kScanSmallMax: at least
// its tile count, and never fewer than for any smaller n (it sizes its tile
// by n, so its tile count alone is not monotone in n).
uint64_t scan_small_descriptors(uint64_t n);
// Descriptors the plain scan's size query asks for: non-decreasing in n, so
// scratch sized for the largest n serves every smaller one.
inline uint64_t scan_tiles(uint64_t n) {
    return n <= kScanSmallMax ? scan_small_descriptors(n)
                              : (n + scan_tile_elems() - 1) / scan_tile_elems();
}
// One launch of the plain scan (the scratch has already been cleared); picks
// the kernel by n as above.
cudaError_t launch_scan(dwp_op op, bool inclusive, const void *in, void *out, uint64_t n,
                        void *scratch, cudaStream_t stream);
cudaError_t launch_scan_small(dwp_op op, bool inclusive, const void *in, void *out, uint64_t n,
                              void *scratch, cudaStream_t stream, const LaunchKnobs &fault);

// Elements per tile of the segmented scan kernel.
uint32_t segscan_tile_elems();
// One launch of the segmented u32 scan (scratch already cleared; nseg >= 1).
cudaError_t launch_segscan(const uint32_t *values, const uint32_t *offsets, uint32_t nseg,
                           uint32_t *out, uint64_t n, bool inclusive, void *scratch,
                           cudaStream_t stream);

// Records per tile of the compaction kernel.
uint32_t compact_tile_records();
// One launch of the stable compaction (scratch already cleared; n >= 1).
cudaError_t launch_compact(const void *records, const uint8_t *flags, uint64_t n, void *out,
                           uint32_t *count, void *scratch, cudaStream_t stream);

// Largest n and elements per block of the two-level (three-launch) scan.
uint64_t two_level_max_n();
uint32_t two_level_chunk();
// The three launches of the two-level scan; the scratch holds the 128-byte
// header and then one u32 total per block.
cudaError_t launch_two_level(dwp_op op, bool inclusive, const void *in, void *out, uint64_t n,
                             void *scratch, cudaStream_t stream);

// Rows per tile of the segmented reduction kernel.
uint32_t segreduce_tile_elems();
// One launch of the segmented u32 reduction (out already cleared, scratch
// header cleared; nseg >= 1, n >= 1).
cudaError_t launch_segreduce(const uint32_t *values, const uint32_t *offsets, uint32_t nseg,
                             uint32_t *out, uint64_t n, void *scratch, cudaStream_t stream);

// Elements per tile of the linear-recurrence kernel.
uint32_t recurrence_tile_elems();
// One launch of the f32 linear recurrence h[t] = a[t] h[t-1] + b[t]
// (scratch already cleared: header + 16 bytes per tile; n >= 1).
cudaError_t launch_recurrence(const float *a, const float *b, float *h, uint64_t n, bool inclusive,
                              void *scratch, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Sequence operators (conv.cu, norm.cu, selscan.cu, selscan_forward.cuh,
// selscan_backward.cuh, selscan_step.cu).  Strides are in elements.

// Streaming multiprocessors of a GB300.  Scratch sizes follow from it, and a
// size query makes no CUDA call: on a GPU with another count the cuts are
// other than measured, and nothing else.
constexpr int kSMs = 152;

struct ConvParams {
    int64_t channels, batch, rows, strips;  // strips: blocks of rows per batch entry
    int width, silu;
    bool weight_f32, weight_wide;  // wide: weight starts on 16 bytes
    const void *x, *weight, *bias, *initial_state;
    void *y, *final_state;
    int64_t x_batch, x_row, y_batch, y_row;
    const uint32_t *offsets;
    uint32_t num_segments;
};
struct ConvBackwardParams {
    ConvParams c;
    int64_t strip_rows;
    const void *grad_out, *grad_final;
    void *grad_x, *grad_initial;
    int64_t grad_batch, grad_row, gx_batch, gx_row;
    float *partial;  // [batch * strips][width + 1][channels]
};
struct ConvStepParams {
    int64_t channels, batch, num_slots;
    int width, silu;
    bool weight_f32, weight_wide;
    const void *x, *weight, *bias;
    void *y, *state;
    int64_t x_row, y_row, state_slot;
    const int32_t *slots;
};
int64_t conv_strip_rows();
cudaError_t launch_conv(dwp_dtype t, const ConvParams &p, bool vec, cudaStream_t s);
cudaError_t launch_conv_backward(dwp_dtype t, const ConvBackwardParams &p, bool vec, cudaStream_t s);
cudaError_t launch_conv_step(dwp_dtype t, const ConvStepParams &p, bool vec, cudaStream_t s);
// Empty segments (all, if offsets is NULL) hand `count` state elements on.
cudaError_t launch_empty_states(dwp_dtype t, const uint32_t *offsets, int64_t segments, int64_t count,
                                const void *src, void *dst, cudaStream_t s);

// Where column sums go: columns [0, end[0]) to out[0], up to end[1] to out[1],
// up to end[2] to out[2] (a NULL out drops its columns).  The first range is
// `planes` planes of equal length, written interleaved.
struct ColumnOut {
    float *out[3];
    int64_t end[3];
    int64_t planes;
};
cudaError_t launch_column_sums(const float *part, int64_t blocks, int64_t cols, const ColumnOut &o,
                               cudaStream_t s);

struct ScanParams {
    int64_t channels, group, groups, batch, rows;  // group: channels of a group
    int64_t chunk_rows, chunks, tiles;             // tiles: saved states per batch entry
    int states, softplus;
    uint32_t group_blocks;  // channel blocks of a group (set by the launcher)
    const void *u, *dt, *z, *B, *C;
    void *out;
    int64_t u_batch, u_row, dt_batch, dt_row, z_batch, z_row, out_batch, out_row;
    int64_t b_batch, b_row, b_group, c_batch, c_row, c_group;
    const float *A, *D, *dt_bias, *initial;
    float *final, *checkpoints;
    const uint32_t *segmap;  // NULL, or a code word per packed row
    bool wide;         // two neighbouring channels, and four neighbouring states of B and C, are one aligned access
    bool states_wide;  // four neighbouring states of A and every state array are one aligned access
    // [batch * (chunks - 1)]: last states, sums of delta per channel, whether a segment began
    float *carry, *carry_sum;
    uint32_t *carry_head;
};
struct ScanBackwardParams {
    ScanParams f;
    const void *grad_out;
    int64_t grad_batch, grad_row;
    const float *grad_final;
    void *grad_u, *grad_dt, *grad_z, *grad_B, *grad_C;
    float *grad_initial;
    float *partial;     // [batch * chunks][channels * (states + 2)]
    float *partial_bc;  // [channel blocks of a group][batch * rows][groups][2][states]
};
struct ScanStepParams {
    int64_t channels, group, groups, batch, num_slots;
    int states, softplus;
    uint32_t group_blocks;
    const void *u, *dt, *z, *B, *C;
    void *out;
    int64_t u_row, dt_row, z_row, out_row, b_row, b_group, c_row, c_group;
    const float *A, *D, *dt_bias;
    float *state;
    int64_t state_slot;
    const int32_t *slots;
    bool wide;  // four neighbouring states of A, B, C and the state are one aligned access
};
// Warps an SM that the gradient's chunks are made for: three times the eight
// that it holds at once (255 registers a lane), so that the last ones to run
// are a small part.  Training step of 2 x 2048 rows x 4096 channels: made for
// eight 780 us, 16 755, 24 715, 56 694 (in 3.5 times the scratch).
constexpr int kScanBackWarpsPerSM = 24;
// Channels one warp of the gradient covers.
int64_t scan_block_channels(int64_t states);
// Warps of the forward that an SM holds (at 168 registers a lane).
constexpr int kScanWarpsPerSM = 12;
// Channels one warp of the forward covers.
int64_t scan_warp_channels(int64_t states);
cudaError_t launch_segment_map(const uint32_t *offsets, uint32_t nseg, uint32_t rows, uint32_t *map,
                               cudaStream_t s);
cudaError_t launch_selscan(dwp_dtype t, const ScanParams &p, cudaStream_t s);
cudaError_t launch_selscan_f32(const ScanParams &p, cudaStream_t s);
cudaError_t launch_selscan_bf16(const ScanParams &p, cudaStream_t s);
cudaError_t launch_selscan_f16(const ScanParams &p, cudaStream_t s);
// States carried over the chunks of the forward.
cudaError_t launch_carry(const ScanParams &p, cudaStream_t s);
cudaError_t launch_selscan_backward(dwp_dtype t, const ScanBackwardParams &p, cudaStream_t s);
cudaError_t launch_selscan_backward_f32(const ScanBackwardParams &p, cudaStream_t s);
cudaError_t launch_selscan_backward_bf16(const ScanBackwardParams &p, cudaStream_t s);
cudaError_t launch_selscan_backward_f16(const ScanBackwardParams &p, cudaStream_t s);
// The gradient's recurrence over the chunks, from the last (chunk 0 of the
// carry) to the second.
cudaError_t launch_scan_walk_back(dwp_dtype t, const ScanParams &p, cudaStream_t s);
cudaError_t launch_scan_walk_back_f32(const ScanParams &p, cudaStream_t s);
cudaError_t launch_scan_walk_back_bf16(const ScanParams &p, cudaStream_t s);
cudaError_t launch_scan_walk_back_f16(const ScanParams &p, cudaStream_t s);
cudaError_t launch_selscan_step(dwp_dtype t, const ScanStepParams &p, cudaStream_t s);

struct NormParams {
    int64_t channels, group, groups, rows;  // group: elements normed together
    float eps;
    int gate_after;
    bool weight_f32, residual_f32;
    const void *x, *residual, *gate, *weight, *scale;
    void *y, *sum;
    int64_t x_row, residual_row, gate_row, y_row, sum_row;
};
struct NormBackwardParams {
    NormParams n;
    int64_t blocks;  // blocks a group's rows are spread over
    const void *v, *x_in, *grad_out, *grad_sum;  // v: the norm's input; x_in: x, for the scale's gradient
    bool v_f32;
    void *grad_x, *grad_residual, *grad_gate;
    int64_t v_row, xin_row, grad_row, gsum_row, gx_row, gres_row, ggate_row;
    float *partial;  // [blocks][1 or 2][channels]
};
cudaError_t launch_norm(dwp_dtype t, const NormParams &p, bool vec, cudaStream_t s);
// Threads of one block of the gradient.
int64_t norm_backward_threads(dwp_dtype t, int64_t group, bool vec);
cudaError_t launch_norm_backward(dwp_dtype t, const NormBackwardParams &p, bool vec, cudaStream_t s);

}  // namespace dwp
