/*
 * dwp.h - device-wide single-pass prefix scan for NVIDIA GB300 (sm_103a).
 *
 * C ABI.  Every entry point takes plain device pointers and sizes, runs as
 * one stream-ordered launch sequence on the caller's stream and returns
 * without synchronising.  The library never allocates memory: the caller
 * owns inputs, outputs and scratch.
 *
 * Operation ("Parallel Prefix Sum (Scan), in depth", section "Inclusive,
 * exclusive and associative"): for an associative operator (+) with identity
 * e, the inclusive scan is y[i] = x[0] (+) ... (+) x[i]; the exclusive scan
 * is y[0] = e and y[i] = x[0] (+) ... (+) x[i-1].  Identities ("Prefix scans
 * and compaction", section "Inclusive and exclusive scan"): 0 for addition,
 * the lowest representable value (0 for u32) for a maximum.
 *
 * Method ("Single-Pass Prefix Scan with Decoupled Look-Back", sections
 * "Three states in a per-block descriptor" and "The publication protocol in
 * code"; "Parallel Prefix Sum (Scan), in depth", section "Scanning a whole
 * array: three grid strategies"): one pass over the data.  Tiles take their
 * index from an atomic counter, publish their aggregate in a 64-bit
 * descriptor (state and value in one word), look back over their
 * predecessors' descriptors until an inclusive prefix is found, publish
 * their own inclusive prefix and write their output.
 *
 * Scratch (two-call pattern, "Parallel Prefix Sum (Scan), in depth",
 * section "Use the library"): call once with d_scratch == NULL to receive
 * the required byte count in *scratch_bytes, then again with a device
 * buffer of at least that many bytes.  The scratch holds the tile counter,
 * a device-side status word and one 8-byte descriptor per tile; each call
 * clears the part it uses with a cudaMemsetAsync on `stream` before its
 * kernel.  Calls that share one scratch buffer must be ordered (same stream
 * or synchronised); overlapping calls on one scratch buffer race.
 *
 * Pointers: every data pointer and the scratch pointer must be 16-byte
 * aligned (DWP_ERR_MISALIGNED otherwise).  Sizes: n < 2^32.
 *
 * Errors: argument errors are reported before anything is enqueued.  A
 * launch error is DWP_ERR_CUDA.  Errors that arise on the device (a
 * look-back or pipeline wait that ran past its limit) are recorded in the
 * scratch status word and returned by dwp_read_status().  All device-side
 * waits are bounded: a kernel never hangs, it records an error and exits.
 */
#ifndef DWP_H
#define DWP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A CUDA stream handle; the same value as a cudaStream_t.  NULL means the
 * legacy default stream. */
typedef struct CUstream_st *dwp_stream;

typedef enum dwp_status {
    DWP_SUCCESS = 0,
    DWP_ERR_INVALID_VALUE = 1,     /* null pointer with n > 0, unknown op/mode, n >= 2^32 */
    DWP_ERR_MISALIGNED = 2,        /* a pointer is not 16-byte aligned */
    DWP_ERR_ALIASING = 3,          /* input, output or scratch ranges overlap (see each call) */
    DWP_ERR_SCRATCH_TOO_SMALL = 4, /* *scratch_bytes is below the size query's answer */
    DWP_ERR_CUDA = 5,              /* a CUDA runtime call or launch failed */
    DWP_ERR_LOOKBACK_TIMEOUT = 6,  /* device: a look-back spin ran past its limit */
    DWP_ERR_PIPELINE_TIMEOUT = 7,  /* device: a shared-memory pipeline wait ran past its limit */
    DWP_ERR_NO_DEVICE = 8,         /* no usable CUDA device */
    DWP_ERR_BOUNDS = 9             /* device, debug bounds build only: an access would have
                                      left its buffer and was skipped (never in the default build) */
} dwp_status;

/* Associative operators of the plain scans. */
typedef enum dwp_op {
    DWP_U32_ADD = 0, /* uint32 addition, wraps modulo 2^32; identity 0 */
    DWP_F32_ADD = 1, /* float32 addition in f32 arithmetic; identity +0.0f */
    DWP_U32_MAX = 2  /* uint32 maximum; identity 0 */
} dwp_op;

typedef enum dwp_mode {
    DWP_EXCLUSIVE = 0,
    DWP_INCLUSIVE = 1
} dwp_mode;

/*
 * Exclusive scan of n elements of d_in (uint32 or float32 per `op`) into
 * d_out.  Definition: "Parallel Prefix Sum (Scan), in depth", section
 * "Inclusive, exclusive and associative"; y[0] is the identity.
 *   op            DWP_U32_ADD, DWP_F32_ADD or DWP_U32_MAX
 *   d_in, d_out   device arrays of n 4-byte elements, contiguous.
 *                 d_out == d_in (exact in-place) is allowed; any other
 *                 overlap is DWP_ERR_ALIASING.
 *   n             element count, 0 <= n < 2^32; n == 0 enqueues only the
 *                 scratch clear.
 *   d_scratch     NULL for the size query, else a device buffer that does
 *                 not overlap d_in or d_out.
 *   scratch_bytes in: size of d_scratch; out (size query): size needed.
 *   stream        stream the work is enqueued on.
 * f32 results are not bit-reproducible from run to run: the grouping of the
 * partial sums depends on look-back timing ("Single-Pass Prefix Scan with
 * Decoupled Look-Back", section "When not to use it").
 */
dwp_status dwp_scan_exclusive(dwp_op op, const void *d_in, void *d_out, size_t n,
                              void *d_scratch, size_t *scratch_bytes, dwp_stream stream);

/* Inclusive scan; arguments as dwp_scan_exclusive.  y[i] includes x[i]. */
dwp_status dwp_scan_inclusive(dwp_op op, const void *d_in, void *d_out, size_t n,
                              void *d_scratch, size_t *scratch_bytes, dwp_stream stream);

/*
 * Segmented uint32 addition scan over CSR offsets ("GPUSegmentedScan",
 * sections "Prefix scans and segmented scans", "Contract" and
 * "Limitations"; "Parallel Prefix Sum (Scan), in depth", section "What scan
 * builds": the running total restarts at every segment boundary).
 *   d_values      device uint32[n], 16-byte aligned
 *   d_offsets     device uint32[num_segments + 1], 4-byte aligned; segment
 *                 s is rows [d_offsets[s], d_offsets[s+1]).  Offsets are
 *                 trusted: non-decreasing with d_offsets[num_segments] <= n
 *                 is a precondition the device does not check (no
 *                 readback); broken offsets give unspecified values but no
 *                 access out of range.  Repeated offsets are empty
 *                 segments and write no rows.
 *   num_segments  N, 0 <= N < 2^32 - 1 (N + 1 offsets are read).
 *   d_out         device uint32[n], 16-byte aligned.  Rows outside
 *                 [d_offsets[0], min(d_offsets[N], n)) are left unwritten.
 *                 Overlap with d_values, d_offsets or d_scratch is
 *                 DWP_ERR_ALIASING.
 *   n             row count, 0 <= n < 2^32.
 *   mode          DWP_EXCLUSIVE (a segment's first row is 0) or
 *                 DWP_INCLUSIVE.
 *   d_scratch, scratch_bytes, stream: as dwp_scan_exclusive (the size
 *                 query depends on n only).
 * u32 sums wrap modulo 2^32.  Results are bit-exact and deterministic.
 */
dwp_status dwp_segmented_scan_u32(const uint32_t *d_values, const uint32_t *d_offsets,
                                  size_t num_segments, uint32_t *d_out, size_t n,
                                  dwp_mode mode, void *d_scratch, size_t *scratch_bytes,
                                  dwp_stream stream);

/*
 * Stable stream compaction of 16-byte records by byte flags ("Prefix scans
 * and compaction", sections "Scan as an index generator" and "Worked
 * example: Stable stream compaction"; "Parallel Prefix Sum (Scan), in
 * depth", section "What scan builds").  Record i is kept when d_flags[i] is
 * nonzero and is written to slot (number of kept records before i) of
 * d_out, so kept records keep their input order; the number kept goes to
 * *d_count.
 *   d_records     device array of n records of 16 bytes each (opaque,
 *                 copied bit for bit), 16-byte aligned
 *   d_flags       device uint8[n], 16-byte aligned
 *   n             record count, 0 <= n < 2^32
 *   d_out         device array with room for n records, 16-byte aligned;
 *                 slots at and past the kept count are left unwritten.
 *   d_count       device uint32, 4-byte aligned: receives the kept count
 *                 (0 for n == 0).
 *   d_scratch, scratch_bytes, stream: as dwp_scan_exclusive.
 * Any overlap among d_out, d_count, d_scratch and the inputs is
 * DWP_ERR_ALIASING.  Results are bit-exact and deterministic.
 */
dwp_status dwp_compact_by_flags(const void *d_records, const uint8_t *d_flags, size_t n,
                                void *d_out, uint32_t *d_count, void *d_scratch,
                                size_t *scratch_bytes, dwp_stream stream);

/*
 * Scan for callers that cannot allocate device memory.  The source pages
 * have no counterpart to this entry point; it is a convenience of this
 * library.  Code that runs inside another framework's allocator hooks or
 * memory-pool callbacks (where cudaMalloc would re-enter that allocator),
 * or a plug-in whose host application owns all device memory, cannot hand
 * the other scan calls a scratch buffer.  This call uses instead a fixed
 * array of about 512 KiB that is part of the library's device image: every
 * GPU that loads libdwp.so holds it until the process exits.  The call
 * itself allocates and frees nothing.
 *   op, d_in, d_out, stream: as dwp_scan_exclusive.
 *   mode      DWP_EXCLUSIVE or DWP_INCLUSIVE.
 *   n         0 <= n <= DWP_SCAN_STATIC_MAX_N (2^28 elements); a larger n
 *             returns DWP_ERR_SCRATCH_TOO_SMALL before anything is enqueued.
 * Every call looks up the current device's address of the array
 * (cudaGetSymbolAddress), so the address stays right after a device or
 * context reset.  The first call on a device also loads the library's
 * device code there: make that first call before any stream capture.  Every
 * call on a device shares the one array, and each call clears the part it
 * uses on `stream` first, so calls must be ordered on the GPU: two calls
 * that overlap on the GPU (different streams, not synchronised) race and
 * give wrong results.  Device-side timeouts are recorded in the array's
 * status word: read it with dwp_read_static_status.  DWP_ERR_NO_DEVICE if
 * there is no current device; otherwise the errors of dwp_scan_exclusive.
 */
#define DWP_SCAN_STATIC_MAX_N 268435456u
dwp_status dwp_scan_static_scratch(dwp_op op, dwp_mode mode, const void *d_in, void *d_out,
                                   size_t n, dwp_stream stream);

/*
 * Device-side status of the most recent dwp_scan_static_scratch call on the
 * current device: what dwp_read_status returns for a caller-owned scratch
 * buffer, read from the built-in array.  Synchronises `stream` (order it
 * after the call).  Copies into host memory only; allocates nothing.
 */
dwp_status dwp_read_static_status(dwp_stream stream);

/*
 * The same scans as dwp_scan_exclusive / dwp_scan_inclusive (`mode` picks
 * one) by the two-level form in three launches: block totals, a one-block
 * scan of the totals, then each block scans its chunk again from its total
 * ("Single-Pass Prefix Scan with Decoupled Look-Back", sections "The
 * two-level decomposition" and "When not to use it").  No descriptors and
 * no spinning; the input is read twice.  For small inputs and for
 * comparison with the single-pass scan.
 *   n            at most 2^26 (DWP_ERR_INVALID_VALUE above).
 *   d_scratch    NULL: *scratch_bytes receives the size needed (128 bytes
 *                plus 4 bytes per 4096-element block).
 * Pointers, alignment, in-place use and errors as for dwp_scan_exclusive.
 */
dwp_status dwp_scan_two_level(dwp_op op, dwp_mode mode, const void *d_in, void *d_out, size_t n,
                              void *d_scratch, size_t *scratch_bytes, dwp_stream stream);

/*
 * Stable compaction in three stages, for comparison with the fused
 * dwp_compact_by_flags ("Prefix scans and compaction", section "Worked
 * example: Stable stream compaction": compare an implementation that
 * materialises the flags and their prefixes with a fused one; section
 * "Common errors": the cost of materialising predicates and prefixes).
 * Same arguments, output and count as dwp_compact_by_flags; the output is
 * bit for bit the same.  The stages, in three launches plus the scan's
 * scratch clear: u32 flags f[i] = (d_flags[i] != 0) written to scratch;
 * dwp_scan_exclusive of f into offsets in scratch; a scatter that reads f,
 * the offsets and each kept record and writes it to its slot.  Memory
 * traffic is about 21 bytes per record plus the kept records' sectors and
 * output, against 17 plus the output for the fused kernel.
 *   d_scratch  NULL: *scratch_bytes receives the size needed (the scan's
 *              scratch plus 8 bytes per record).  Otherwise at least that
 *              many bytes, 16-byte aligned, overlapping no other argument;
 *              dwp_read_status on it reports the scan's device status.
 * Errors as for dwp_compact_by_flags.
 */
dwp_status dwp_compact_by_flags_staged(const void *d_records, const uint8_t *d_flags, size_t n,
                                       void *d_out, uint32_t *d_count, void *d_scratch,
                                       size_t *scratch_bytes, dwp_stream stream);

/*
 * Segmented u32 addition reduction over CSR offsets ("GPUSegmentedScan"
 * (luma.gl), section "Composition", which names the segmented reduction
 * beside the segmented scan; the segments are those of "Contract"):
 * d_out[s] = d_values[offsets[s]] + ... + d_values[offsets[s+1] - 1],
 * wrapping modulo 2^32, and 0 for an empty segment.
 *   d_values     n u32 (device, 16-byte aligned).
 *   d_offsets    num_segments + 1 u32 (device, 4-byte aligned),
 *                non-decreasing, d_offsets[num_segments] <= n.  Trusted, as
 *                for dwp_segmented_scan_u32: other offsets give unspecified
 *                sums, but every access stays inside the arrays.
 *   d_out        num_segments u32 (device, 4-byte aligned), overlapping no
 *                other argument.
 *   d_scratch    NULL: *scratch_bytes receives the size needed (128 bytes:
 *                a tile counter and the status word; this operation keeps
 *                no per-tile state).  Otherwise at least that many bytes,
 *                16-byte aligned, overlapping no other argument.
 * The call clears d_out and the scratch on `stream` and launches one kernel;
 * n == 0 or num_segments == 0 launches nothing.  Segment pieces that cross a
 * tile edge are added with atomics: the result is exact (u32 addition wraps
 * and commutes) and does not depend on the order.  Errors as for
 * dwp_segmented_scan_u32.
 */
dwp_status dwp_segmented_reduce_u32(const uint32_t *d_values, const uint32_t *d_offsets,
                                    size_t num_segments, uint32_t *d_out, size_t n,
                                    void *d_scratch, size_t *scratch_bytes, dwp_stream stream);

/*
 * First-order linear recurrence ("Parallel Prefix Sum (Scan), in depth",
 * section "What scan builds"): h[t] = a[t] * h[t-1] + b[t] with h[-1] = 0,
 * computed as a single-pass scan of the pairs (a[t], b[t]) under
 * (a1, b1) then (a2, b2) = (a1 a2, a2 b1 + b2).
 *   d_a, d_b  n f32 coefficients and inputs (device, 16-byte aligned).
 *   d_h       n f32 outputs (device, 16-byte aligned).  DWP_INCLUSIVE
 *             writes h[t]; DWP_EXCLUSIVE writes the state before step t,
 *             h[t-1] (0 at t = 0).  d_h may equal d_a or d_b exactly (in
 *             place); any other overlap with them is DWP_ERR_ALIASING.
 *   d_scratch NULL: *scratch_bytes receives the size needed (a 128-byte
 *             header plus 16 bytes per tile) and nothing else happens.
 *             Otherwise at least that many bytes, 16-byte aligned, owned by
 *             the caller, overlapping no other argument.
 * Arithmetic is f32 with one fused multiply-add per step; the grouping
 * differs from the sequential loop, so results agree with it to f32
 * rounding, not bit for bit.  Errors as for dwp_scan_exclusive; the
 * Decoupled Fallback applies except in place.
 */
dwp_status dwp_linear_recurrence_f32(const float *d_a, const float *d_b, float *d_h, size_t n,
                                     dwp_mode mode, void *d_scratch, size_t *scratch_bytes,
                                     dwp_stream stream);

/*
 * Sequence operators.
 *
 * The linear recurrence above in the form a state space layer uses it, with
 * what stands around it there: the short causal convolution before it, the
 * selective scan, and the norm around the block; the recurrence with a matrix
 * state, the gated delta rule, and the layer norm; each with its gradient, and
 * the convolution and the recurrences with a form for single tokens.
 *
 * Layout.  Rows are tokens; a row's channels are contiguous.  A tensor of
 * rows is [batch, rows, channels], given by its address, batch stride and row
 * stride, in elements: a column range of a wider tensor (half of a
 * projection's output) needs no copy.  With `offsets` the batch is 1 and the
 * rows are num_segments sequences packed one after another, by CSR offsets as
 * for dwp_segmented_scan_u32: uint32[num_segments + 1], non-decreasing, empty
 * segments allowed, trusted (other offsets give unspecified values but no
 * access out of range); rows outside [offsets[0], offsets[num_segments]) are
 * left unwritten in every output and add nothing to any sum.  Without it each
 * batch entry is one sequence.  "Sequence s" below is segment s or batch
 * entry s, and the number of sequences is num_segments or batch.
 *
 * Types.  Activations have one type per call (dwp_dtype).  Arithmetic, sums,
 * norms and states of the scan are f32; an activation is rounded once, when
 * it is written.
 *
 * Pointers need their element's alignment only.  Rows that start on 16-byte
 * boundaries (address, strides and channel count) take wider accesses.
 *
 * Outputs overlap neither inputs nor one another nor the scratch
 * (DWP_ERR_ALIASING), except where a call says so; column ranges of one wider
 * tensor that share no element do not overlap.  Sizes: batch * rows < 2^31,
 * at most 2^17 channels, 1024 groups and 2^30 - 2 segments, strides up to 2^40
 * elements, 2^58 elements from a tensor's first row to its last.
 * DWP_ERR_INVALID_VALUE for a NULL required pointer, a size, stride or type out
 * of range, or a stride below the row it spans.
 *
 * These calls keep no status word: no kernel of theirs waits for another, and
 * only the gated delta rule's wait for copies and products of their own, each
 * wait bounded; should one run out, what the block had still to compute is NaN
 * (of a walk along a sequence and head all that it writes).  Results are
 * deterministic, bit for bit from run to run.  Scratch follows the two-call
 * pattern above, 16-byte aligned and never less than 16 bytes; its contents on
 * entry do not matter.
 */
typedef enum dwp_dtype { DWP_F32 = 0, DWP_BF16 = 1, DWP_F16 = 2 } dwp_dtype;

/* Rows of a tensor: element strides between batch entries and rows. */
typedef struct dwp_rows {
    void *data;
    int64_t batch_stride;
    int64_t row_stride;
} dwp_rows;

/*
 * Causal depthwise convolution, per channel:
 *   p[t] = bias + sum_k weight[k] * x[t - (width-1) + k],  out = p, or p * sigmoid(p)
 * where the rows before a sequence's first are its initial state's.
 *   dtype          of x, out and the states; weight_dtype: dtype or DWP_F32,
 *                  of weight and bias
 *   width          1 .. 8
 *   weight         [channels, width];   bias  [channels] or NULL
 *   offsets        NULL, or see above
 *   initial_state  [sequences, width - 1, channels], or NULL for zeros: the
 *                  inputs before each sequence's first row, oldest first
 *   final_state    NULL, or the same for the rows after its last (may not
 *                  overlap initial_state)
 */
typedef struct dwp_conv_args {
    int64_t dtype, weight_dtype, silu, width;
    int64_t channels, batch, rows, num_segments;
    dwp_rows x, out;
    const void *weight, *bias;
    const uint32_t *offsets;
    const void *initial_state;
    void *final_state;
} dwp_conv_args;
dwp_status dwp_causal_conv(const dwp_conv_args *args, dwp_stream stream);

/*
 * Gradient of dwp_causal_conv.
 *   conv                the forward's arguments (out, final_state unused)
 *   grad_out            of the output;  grad_final_state  NULL for zeros
 *   grad_x              of x (dtype)
 *   grad_weight         f32 [channels, width];  grad_bias  f32 [channels] or NULL
 *   grad_initial_state  NULL, or as initial_state
 */
typedef struct dwp_conv_backward_args {
    dwp_conv_args conv;
    dwp_rows grad_out, grad_x;
    const void *grad_final_state;
    float *grad_weight, *grad_bias;
    void *grad_initial_state;
} dwp_conv_backward_args;
dwp_status dwp_causal_conv_backward(const dwp_conv_backward_args *args, void *d_scratch,
                                    size_t *scratch_bytes, dwp_stream stream);

/*
 * dwp_causal_conv for one new row of each of `batch` sequences, the states
 * updated in place.
 *   x, out   [batch, channels] (batch_stride unused)
 *   state    [num_slots, width - 1, channels], slot_stride elements apart
 *   slots    int32[batch]: the slot of each row; a row whose slot lies outside
 *            [0, num_slots) is padding: its output is 0 and no state changes.
 *            NULL: row i has slot i.  No two rows may name one slot.
 */
typedef struct dwp_conv_step_args {
    int64_t dtype, weight_dtype, silu, width;
    int64_t channels, batch, num_slots;
    dwp_rows x, out;
    const void *weight, *bias;
    void *state;
    int64_t slot_stride;
    const int32_t *slots;
} dwp_conv_step_args;
dwp_status dwp_causal_conv_step(const dwp_conv_step_args *args, dwp_stream stream);

/* Rows between the states that the selective scan keeps for its gradient. */
#define DWP_SCAN_CHECKPOINT_ROWS 16

/*
 * Selective state space scan: per channel d (group g) and state n,
 *   delta = dt + dt_bias, through log(1 + exp()) if softplus
 *   h[t]  = exp(delta A[d,n]) h[t-1] + delta u B[t,g,n]
 *   y[t]  = sum_n C[t,g,n] h[t] + D[d] u,   out = y, or y * silu(z)
 *   u, dt, z, out  rows of `channels`; z.data may be NULL
 *   B, C           rows of [groups, states], group_stride elements apart;
 *                  groups divides channels, and channel d has group
 *                  d / (channels / groups)
 *   states         1 .. 128
 *   A              f32 [channels, states];  D, dt_bias  f32 [channels] or NULL
 *   initial_state  f32 [sequences, channels, states], or NULL for zeros
 *   final_state    NULL, or the same after each sequence's last row
 *   checkpoints    NULL, or f32 [batch, ceil(rows / DWP_SCAN_CHECKPOINT_ROWS),
 *                  channels, states]: states kept for the gradient
 */
typedef struct dwp_selective_scan_args {
    int64_t dtype, softplus;
    int64_t channels, states, groups, batch, rows, num_segments;
    dwp_rows u, dt, z, B, C, out;
    int64_t b_group_stride, c_group_stride;
    const float *A, *D, *dt_bias;
    const uint32_t *offsets;
    const float *initial_state;
    float *final_state, *checkpoints;
} dwp_selective_scan_args;
dwp_status dwp_selective_scan(const dwp_selective_scan_args *args, void *d_scratch,
                              size_t *scratch_bytes, dwp_stream stream);

/*
 * Gradient of dwp_selective_scan.
 *   scan        the forward's arguments, checkpoints as the forward wrote them
 *               (out, final_state unused)
 *   grad_out    of the output;  grad_final_state  NULL for zeros
 *   grad_u, grad_dt, grad_z  [batch, rows, channels], dense, dtype (grad_z
 *               NULL without z);  grad_B, grad_C  [batch, rows, groups,
 *               states], dense, dtype
 *   grad_A f32 [channels, states];  grad_D, grad_dt_bias f32 [channels], or
 *               NULL;  grad_initial_state  NULL, or as initial_state
 *   scratch     grows with rows x channels: it holds a share of grad_B and
 *               grad_C, 8 * states bytes, for each row, group and block of the
 *               group's channels, a block being 32 channels at up to 16
 *               states, 16 at up to 32, 8 at up to 64 and 4 above.  That is 4
 *               bytes a row and channel at 16 states, 16 at 32, 64 at 64 and
 *               256 at 128.  Beside it up to 17 MB, or 4 * batch * channels *
 *               (states + 2) bytes where that is more, and 4 bytes a packed row.
 */
typedef struct dwp_selective_scan_backward_args {
    dwp_selective_scan_args scan;
    dwp_rows grad_out;
    const float *grad_final_state;
    void *grad_u, *grad_dt, *grad_z, *grad_B, *grad_C;
    float *grad_A, *grad_D, *grad_dt_bias, *grad_initial_state;
} dwp_selective_scan_backward_args;
dwp_status dwp_selective_scan_backward(const dwp_selective_scan_backward_args *args,
                                       void *d_scratch, size_t *scratch_bytes, dwp_stream stream);

/*
 * dwp_selective_scan for one new row of each of `batch` sequences, the states
 * updated in place; slots as for dwp_causal_conv_step, `state` f32
 * [num_slots, channels, states], slot_stride elements apart.
 */
typedef struct dwp_selective_scan_step_args {
    int64_t dtype, softplus;
    int64_t channels, states, groups, batch, num_slots;
    dwp_rows u, dt, z, B, C, out;
    int64_t b_group_stride, c_group_stride;
    const float *A, *D, *dt_bias;
    float *state;
    int64_t slot_stride;
    const int32_t *slots;
} dwp_selective_scan_step_args;
dwp_status dwp_selective_scan_step(const dwp_selective_scan_step_args *args, dwp_stream stream);

/*
 * Gated delta rule: per head, a state S of keys x values decays and is then
 * corrected toward its new row,
 *   S' = exp(g[t]) S[t-1],  u = beta[t] (v[t] - S'^T k[t])
 *   S[t] = S' + k[t] u^T,   out[t] = scale S[t]^T q[t]
 *   q, k           rows of [key_heads, keys];  v, out  rows of [heads, values].
 *                  key_heads divides heads, and head h has the queries and keys
 *                  of key head h / (heads / key_heads).  For overlap a row
 *                  counts as one piece, from its first head to its last
 *   keys, values   1 .. 128 each;  heads  at most 1024
 *   g              f32 rows of [heads], the log of the decay; data NULL for no
 *                  decay.  Below -110 (-infinity too) it counts as -110, whose
 *                  exponential is 0 in f32 all the same
 *   beta           rows of [heads], beta_dtype: dtype or DWP_F32
 *   scale          finite as an f32
 *   initial_state  f32 [sequences, heads, keys, values], or NULL for zeros
 *   final_state    NULL, or the same after each sequence's last row (may not
 *                  overlap initial_state)
 *   checkpoints    NULL, or what the gradient needs, to be handed on as it is:
 *                  f32 [chunks, heads, DWP_DELTA_CHUNK * (2 * DWP_DELTA_CHUNK
 *                  + values') + keys' * values], 16-byte aligned, keys' and
 *                  values' being rounded up to a multiple of 64; chunks is
 *                  batch * ceil(rows / DWP_DELTA_CHUNK), or with offsets rows /
 *                  DWP_DELTA_CHUNK + num_segments
 *   scratch        without checkpoints 8 * DWP_DELTA_CHUNK^2 bytes for each
 *                  of those chunks and head; beside it up to 30 MB where long
 *                  bf16 batch entries (24 chunks and more) have few heads (under
 *                  51 in all) and are cut in parts
 * A sequence is taken in chunks of DWP_DELTA_CHUNK rows from its first.  A
 * value that is not finite reaches its own sequence and heads only, but there
 * the rows before it in its chunk too: a batch entry that is padded at its end
 * is padded with numbers (zeros, say), never with memory that was not written,
 * or its length is given by offsets, whose rows outside are not read.
 * Products of two f32 numbers (states, corrections, weights q.k, f32 rows) take
 * each in two pieces of bf16, 17 bits together (f32 outputs are 3e-6 to 8e-6
 * off in the 2-norm; the gradients of g and beta, sums that cancel, up to 1.3e-5
 * where they have few rows or keys, of one row and head up to 4e-5; a bf16
 * output by its own rounding, 1.7e-3); beyond 3.38e38, bf16's largest, an f32 is
 * not finite.
 */
#define DWP_DELTA_CHUNK 64
typedef struct dwp_heads {
    void *data;
    int64_t batch_stride, row_stride, head_stride; /* elements */
} dwp_heads;
typedef struct dwp_delta_args {
    int64_t dtype, beta_dtype;
    int64_t keys, values, key_heads, heads, batch, rows, num_segments;
    double scale;
    dwp_heads q, k, v, out;
    dwp_rows g, beta;
    const uint32_t *offsets;
    const float *initial_state;
    float *final_state, *checkpoints;
} dwp_delta_args;
dwp_status dwp_gated_delta_rule(const dwp_delta_args *args, void *d_scratch, size_t *scratch_bytes,
                                dwp_stream stream);

/*
 * Gradient of dwp_gated_delta_rule.
 *   delta         the forward's arguments, checkpoints as the forward wrote
 *                 them (out, final_state unused)
 *   grad_out      of the output;  grad_final_state  NULL for zeros
 *   grad_q, grad_k  [batch, rows, key_heads, keys], grad_v  [batch, rows,
 *                 heads, values], dense, dtype: where heads share a key head,
 *                 the sum over them, rounded once
 *   grad_g        f32 [batch, rows, heads], dense, or NULL (always without g);
 *                 grad_beta  the same, beta_dtype
 *   grad_initial_state  NULL, or as initial_state
 *   scratch       4 * (keys' * values + DWP_DELTA_CHUNK * values') bytes for
 *                 each of the chunks and head; beside it as the forward's
 */
typedef struct dwp_delta_backward_args {
    dwp_delta_args delta;
    dwp_heads grad_out;
    const float *grad_final_state;
    void *grad_q, *grad_k, *grad_v;
    float *grad_g;
    void *grad_beta;
    float *grad_initial_state;
} dwp_delta_backward_args;
dwp_status dwp_gated_delta_rule_backward(const dwp_delta_backward_args *args, void *d_scratch,
                                         size_t *scratch_bytes, dwp_stream stream);

/*
 * dwp_gated_delta_rule for one new row of each of `batch` sequences, the
 * states updated in place; slots as for dwp_causal_conv_step, `state` f32
 * [num_slots, heads, keys, values], slot_stride elements apart.
 */
typedef struct dwp_delta_step_args {
    int64_t dtype, beta_dtype;
    int64_t keys, values, key_heads, heads, batch, num_slots;
    double scale;
    dwp_heads q, k, v, out;
    dwp_rows g, beta;
    float *state;
    int64_t slot_stride;
    const int32_t *slots;
} dwp_delta_step_args;
dwp_status dwp_gated_delta_rule_step(const dwp_delta_step_args *args, dwp_stream stream);

/*
 * Root-mean-square norm around a block, over each of `groups` equal parts of
 * a row of `channels` (channels / groups at most DWP_NORM_MAX_GROUP, rows *
 * groups < 2^31):
 *   v   = residual + scale * x, written to `sum`; or x without a residual
 *   t   = v * silu(gate) (gate given, gate_after 0), else v
 *   out = t / sqrt(mean(t^2) + eps) * weight, times silu(gate) if gate_after
 *   x, gate, out    dtype; gate.data may be NULL.  out may be x exactly.
 *   residual, sum   residual_dtype: dtype or DWP_F32; both or neither.  sum
 *                   may be residual exactly.
 *   weight, scale   [channels], weight_dtype: dtype or DWP_F32; scale NULL
 *                   for 1, and only with a residual
 * Tensors are [rows, channels] (batch_stride unused).
 */
#define DWP_NORM_MAX_GROUP 16384
typedef struct dwp_norm_args {
    int64_t dtype, weight_dtype, residual_dtype, gate_after;
    int64_t channels, groups, rows;
    double eps;
    dwp_rows x, residual, gate, sum, out;
    const void *weight, *scale;
} dwp_norm_args;
dwp_status dwp_block_norm(const dwp_norm_args *args, dwp_stream stream);

/*
 * Gradient of dwp_block_norm.
 *   norm           the forward's arguments: x where scale is given, `sum` as
 *                  the forward wrote it where residual was given (residual
 *                  and out unused)
 *   grad_out       of the output;  grad_sum  of `sum`, residual_dtype, or NULL
 *   grad_x         dtype, or NULL;  grad_residual  residual_dtype, with a
 *                  residual only, or NULL;  grad_gate  dtype, with a gate
 *   grad_weight    f32 [channels];  grad_scale  f32 [channels], with a scale
 */
typedef struct dwp_norm_backward_args {
    dwp_norm_args norm;
    dwp_rows grad_out, grad_sum, grad_x, grad_residual, grad_gate;
    float *grad_weight, *grad_scale;
} dwp_norm_backward_args;
dwp_status dwp_block_norm_backward(const dwp_norm_backward_args *args, void *d_scratch,
                                   size_t *scratch_bytes, dwp_stream stream);

/*
 * Layer norm, over each of `groups` equal parts of a row of `channels`
 * (limits as for dwp_block_norm):
 *   v   = residual + x, written to `sum`; or x without a residual
 *   out = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * weight + bias
 *   x, out          dtype.  out may be x exactly.
 *   residual, sum   residual_dtype: dtype or DWP_F32; both or neither.  sum
 *                   may be residual exactly.
 *   weight, bias    [channels], weight_dtype: dtype or DWP_F32; NULL for ones,
 *                   zeros
 * Tensors are [rows, channels] (batch_stride unused).  Mean and squares about
 * it are kept together, so a mean far from zero costs no accuracy.
 */
typedef struct dwp_layer_norm_args {
    int64_t dtype, weight_dtype, residual_dtype;
    int64_t channels, groups, rows;
    double eps;
    dwp_rows x, residual, sum, out;
    const void *weight, *bias;
} dwp_layer_norm_args;
dwp_status dwp_layer_norm(const dwp_layer_norm_args *args, dwp_stream stream);

/*
 * Gradient of dwp_layer_norm.
 *   norm           the forward's arguments: `sum` as the forward wrote it where
 *                  residual was given, else x (residual, out and bias unused)
 *   grad_out       of the output;  grad_sum  of `sum`, residual_dtype, or NULL
 *   grad_x         dtype, or NULL;  grad_residual  residual_dtype, with a
 *                  residual only, or NULL
 *   grad_weight, grad_bias  f32 [channels], or NULL
 */
typedef struct dwp_layer_norm_backward_args {
    dwp_layer_norm_args norm;
    dwp_rows grad_out, grad_sum, grad_x, grad_residual;
    float *grad_weight, *grad_bias;
} dwp_layer_norm_backward_args;
dwp_status dwp_layer_norm_backward(const dwp_layer_norm_backward_args *args, void *d_scratch,
                                   size_t *scratch_bytes, dwp_stream stream);

/*
 * Device-side status of the most recent call that used d_scratch.
 * Synchronises `stream`, then reads the status word.  Returns DWP_SUCCESS,
 * DWP_ERR_LOOKBACK_TIMEOUT or DWP_ERR_PIPELINE_TIMEOUT (and, in a library
 * built with -DDWP_DEBUG_BOUNDS=1, DWP_ERR_BOUNDS); DWP_ERR_CUDA if the
 * synchronisation or the read fails; DWP_ERR_INVALID_VALUE for NULL.
 */
dwp_status dwp_read_status(const void *d_scratch, dwp_stream stream);

/*
 * Decoupled Fallback count of the most recent call that used d_scratch
 * ("GPU Prefix Sums", section "Decoupled Fallback").  A tile whose
 * look-back waits too long on a predecessor that has not published reduces
 * that predecessor's input itself and publishes the result with a
 * compare-and-swap; *count receives the number of such swaps that won.  It
 * is 0 in a healthy run: the fallback starts only after thousands of polls
 * (milliseconds).  Synchronises `stream`.  DWP_ERR_INVALID_VALUE for a NULL
 * argument; DWP_ERR_CUDA if the synchronisation or the read fails.
 */
dwp_status dwp_read_fallbacks(const void *d_scratch, dwp_stream stream, uint32_t *count);

/*
 * Look-back counters of the most recent call that used d_scratch (plain
 * scan, segmented scan or compaction): Decoupled Fallbacks won (as
 * dwp_read_fallbacks), intermediate descriptors published by a bounded
 * look-back window ("Single-Pass Prefix Scan with Decoupled Look-Back",
 * section "Why the work stays linear"; see dwp_set_lookback_window), and
 * look-back steps that jumped over such an intermediate.  Any output pointer
 * may be NULL.  Synchronises `stream`.  DWP_ERR_INVALID_VALUE for a NULL
 * d_scratch; DWP_ERR_CUDA if the synchronisation or the read fails.
 */
dwp_status dwp_read_lookback_stats(const void *d_scratch, dwp_stream stream, uint32_t *fallbacks,
                                   uint32_t *intermediates, uint32_t *jumps);

/* Static, NUL-terminated name of a status code. */
const char *dwp_status_string(dwp_status status);

/* Library version: major * 10000 + minor * 100 + patch. */
int dwp_version(void);

/*
 * Look-back window, a tuning setting for every later call in this process
 * ("Single-Pass Prefix Scan with Decoupled Look-Back", section "Why the work
 * stays linear"): 0 (the default) lets a look-back follow the chain of
 * predecessors as far as it goes.  tiles > 0 bounds it: each time a tile's
 * look-back has folded `tiles` more predecessors without reaching a prefix,
 * it publishes an intermediate descriptor (the sum so far with its own
 * aggregate, and how many tiles that covers), and a later look-back that
 * meets it jumps over that many tiles at once.  Folds go 32 tiles at a
 * time, so the window is effectively rounded up to a multiple of 32.
 * Applies to the plain and segmented scans and to compaction; results do not
 * depend on it (bit for bit for the integer operations).  Not thread-safe;
 * affects every device.  Always DWP_SUCCESS.
 */
dwp_status dwp_set_lookback_window(uint32_t tiles);

/*
 * Test hook, not for production use.  For every later call in this process
 * until reset:
 *   - the tile with index `never_publish_tile` does its work but never
 *     publishes its descriptor (UINT32_MAX disables this);
 *   - look-back spins give up after `spin_limit` polls (0 restores the
 *     default, about a second of polling);
 *   - a look-back takes the Decoupled Fallback after `fallback_polls` polls
 *     on an unpublished predecessor (0 restores the default, 4096 polls;
 *     UINT32_MAX disables the fallback).
 * With the fallback on, the successors of the silent tile reduce its input
 * themselves and the call succeeds with correct output (see
 * dwp_read_fallbacks).  With it off, or for an in-place scan (where the
 * fallback is always off: the silent tile's input may already have been
 * overwritten), they record DWP_ERR_LOOKBACK_TIMEOUT in the scratch status
 * and exit instead of waiting forever.  Not thread-safe; affects every
 * device.
 */
dwp_status dwp_debug_set_fault(uint32_t never_publish_tile, uint32_t spin_limit,
                               uint32_t fallback_polls);

/*
 * Test hook, not for production use: the step-by-step trace of the warp
 * layer's Hillis-Steele scan ("Parallel Prefix Sum (Scan), in depth",
 * section "Hillis-Steele: short span, too much work"), the shuffle scan that
 * dwp_scan_two_level runs on every warp.  One warp loads d_x[0 .. width)
 * (u32 addition; lanes past width hold 0) and runs the scan; after step k
 * (k = 0..4, offset d = 2^k) lane l writes its running value to
 * d_steps[width * k + l] for l < width.  So the page's 8-element trace can
 * be checked step by step on the device.
 *   d_x      device uint32[width];   d_steps  device uint32[5 * width]
 *   width    1 .. 32 (DWP_ERR_INVALID_VALUE otherwise, or for NULL pointers)
 * Asynchronous on `stream`; DWP_ERR_CUDA if the launch fails.
 */
dwp_status dwp_debug_warp_scan_trace(const uint32_t *d_x, size_t width, uint32_t *d_steps,
                                     dwp_stream stream);

/*
 * Test hook, not for production use: schedule perturbation for every later
 * call of the look-back kernels (plain and segmented scan, compaction,
 * linear recurrence) in this process until reset.  A missing ordering step
 * in a chained scan shows only under rare interleavings ("Parallel Prefix
 * Sum (Scan), in depth", section "Failure modes"); this makes a seeded
 * subset of tiles sleep at their publication points (after drawing the
 * tile index, before publishing the aggregate, before the look-back, before
 * publishing the prefix, and between the two words of a two-word
 * descriptor), so that descriptors appear in other orders than the
 * hardware's usual one.  Results must not change.
 *   seed          selects the subset and the sleep lengths
 *   fraction_ppm  share of (tile, point) pairs that sleep, in parts per
 *                 million (0 switches the hook off; at most 1000000)
 *   max_ns        longest sleep, at most 100000 ns
 * Every sleep is bounded.  DWP_ERR_INVALID_VALUE for arguments out of
 * range.  Not thread-safe; affects every device.
 */
dwp_status dwp_debug_set_delay(uint32_t seed, uint32_t fraction_ppm, uint32_t max_ns);

#ifdef __cplusplus
}
#endif

#endif /* DWP_H */
