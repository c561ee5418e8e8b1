// C entry points of the sequence operators: argument validation, the scratch
// size query and the launches.  As in api.cu, validation happens before any
// CUDA call.
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "launch.h"
#include "sequence_check.h"

namespace {

using namespace dwp;

// ---------------------------------------------------------------------------
// causal convolution

int64_t check_conv(Check &c, const dwp_conv_args &a, bool backward) {
    c.require(dtype_ok(a.dtype) && (a.weight_dtype == a.dtype || a.weight_dtype == DWP_F32) && a.width >= 1 &&
              a.width <= kMaxWidth && (a.silu == 0 || a.silu == 1));
    const int64_t seqs = sequences(c, a.channels, a.batch, a.rows, a.num_segments, a.offsets);
    if (c.status != DWP_SUCCESS) return 0;
    const int64_t halo = a.width - 1;
    if (a.batch * a.rows > 0) {
        c.rows(a.x, a.dtype, a.batch, a.rows, a.channels, false);
        if (!backward) c.rows(a.out, a.dtype, a.batch, a.rows, a.channels, true);
    }
    c.dense(a.weight, a.weight_dtype, a.channels * a.width, false, false);
    c.dense(a.bias, a.weight_dtype, a.channels, false, true);
    c.dense(a.initial_state, a.dtype, seqs * halo * a.channels, false, true, &c.bits);
    if (!backward) c.dense(a.final_state, a.dtype, seqs * halo * a.channels, true, true, &c.bits);
    return seqs;
}

ConvParams conv_params(const dwp_conv_args &a, int64_t strip) {
    ConvParams p = {};
    p.channels = a.channels, p.batch = a.batch, p.rows = a.rows, p.strips = ceil_div(a.rows, strip);
    p.width = int(a.width), p.silu = int(a.silu), p.weight_f32 = a.weight_dtype == DWP_F32;
    p.weight_wide = aligned(a.weight, 16);
    p.x = a.x.data, p.weight = a.weight, p.bias = a.bias;
    p.initial_state = a.initial_state, p.final_state = a.final_state;
    p.y = a.out.data;
    p.x_batch = a.x.batch_stride, p.x_row = a.x.row_stride;
    p.y_batch = a.out.batch_stride, p.y_row = a.out.row_stride;
    p.offsets = a.offsets, p.num_segments = uint32_t(a.num_segments);
    return p;
}

dwp_status conv_forward(const dwp_conv_args &a, cudaStream_t s) {
    Check c;
    const int64_t seqs = check_conv(c, a, false);
    if (c.status != DWP_SUCCESS) return c.status;
    if (c.regions.clash()) return DWP_ERR_ALIASING;
    const auto t = static_cast<dwp_dtype>(a.dtype);
    const int64_t count = (a.width - 1) * a.channels;
    if (a.final_state && (a.offsets || a.rows == 0)) {
        const cudaError_t err = launch_empty_states(t, a.offsets, seqs, count, a.initial_state, a.final_state, s);
        if (err != cudaSuccess) return launched(err);
    }
    if (a.batch * a.rows == 0 || seqs == 0) return DWP_SUCCESS;
    return launched(launch_conv(t, conv_params(a, conv_strip_rows()), c.wide(a.channels, a.dtype), s));
}

// Rows of a strip of the gradient: long enough that the taps' partial sums
// are a small share of the traffic.
constexpr int64_t kGradStrip = 64;

dwp_status conv_backward(const dwp_conv_backward_args &a, void *scratch, size_t *bytes, cudaStream_t s) {
    Check c;
    const dwp_conv_args &f = a.conv;
    const int64_t seqs = check_conv(c, f, true);
    const int64_t halo = f.width - 1;
    dwp_status st = c.status;
    if (st != DWP_SUCCESS) return st;
    const int64_t n = f.batch * f.rows;
    if (n > 0) {
        c.rows(a.grad_out, f.dtype, f.batch, f.rows, f.channels, false);
        c.rows(a.grad_x, f.dtype, f.batch, f.rows, f.channels, true);
    }
    c.dense(a.grad_final_state, f.dtype, seqs * halo * f.channels, false, true, &c.bits);
    c.dense(a.grad_initial_state, f.dtype, seqs * halo * f.channels, true, true, &c.bits);
    c.dense(a.grad_weight, DWP_F32, f.channels * f.width, true, false);
    c.dense(a.grad_bias, DWP_F32, f.channels, true, true);
    const int64_t strips = ceil_div(f.rows, kGradStrip);
    const size_t need = round16(size_t(f.batch * strips * (f.width + 1) * f.channels) * 4u);
    if (!c.scratch(scratch, bytes, need, &st)) return st;
    const auto t = static_cast<dwp_dtype>(f.dtype);
    if (a.grad_initial_state && (f.offsets || f.rows == 0)) {
        const cudaError_t err = launch_empty_states(t, f.offsets, seqs, halo * f.channels, a.grad_final_state,
                                                    a.grad_initial_state, s);
        if (err != cudaSuccess) return launched(err);
    }
    if (n == 0 || seqs == 0)
        return launched(launch_clear(a.grad_weight, size_t(f.channels * f.width) * 4u, a.grad_bias,
                                     size_t(f.channels) * 4u, s));
    ConvBackwardParams p = {};
    p.c = conv_params(f, kGradStrip);
    p.strip_rows = kGradStrip;
    p.grad_out = a.grad_out.data, p.grad_batch = a.grad_out.batch_stride, p.grad_row = a.grad_out.row_stride;
    p.grad_x = a.grad_x.data, p.gx_batch = a.grad_x.batch_stride, p.gx_row = a.grad_x.row_stride;
    p.grad_final = a.grad_final_state, p.grad_initial = a.grad_initial_state;
    p.partial = static_cast<float *>(scratch);
    cudaError_t err = launch_conv_backward(t, p, c.wide(f.channels, f.dtype), s);
    if (err != cudaSuccess) return launched(err);
    const ColumnOut o{{a.grad_weight, a.grad_bias, nullptr},
                      {f.channels * f.width, f.channels * (f.width + 1), 0},
                      f.width};
    return launched(launch_column_sums(p.partial, f.batch * strips, f.channels * (f.width + 1), o, s));
}

dwp_status conv_step(const dwp_conv_step_args &a, cudaStream_t s) {
    Check c;
    c.require(dtype_ok(a.dtype) && (a.weight_dtype == a.dtype || a.weight_dtype == DWP_F32) && a.width >= 1 &&
              a.width <= kMaxWidth && (a.silu == 0 || a.silu == 1) && a.channels >= 1 &&
              a.channels <= kMaxChannels && a.batch >= 0 && a.batch <= kMaxRows);
    if (c.status != DWP_SUCCESS) return c.status;
    if (a.batch == 0) return DWP_SUCCESS;
    c.rows(a.x, a.dtype, 1, a.batch, a.channels, false);
    c.rows(a.out, a.dtype, 1, a.batch, a.channels, true);
    c.dense(a.weight, a.weight_dtype, a.channels * a.width, false, false);
    c.dense(a.bias, a.weight_dtype, a.channels, false, true);
    check_slots(c, a.state, a.dtype, a.batch, a.num_slots, a.slot_stride, (a.width - 1) * a.channels, a.slots);
    if (c.status != DWP_SUCCESS) return c.status;
    if (c.regions.clash()) return DWP_ERR_ALIASING;
    ConvStepParams p = {};
    p.channels = a.channels, p.batch = a.batch, p.num_slots = a.num_slots;
    p.width = int(a.width), p.silu = int(a.silu), p.weight_f32 = a.weight_dtype == DWP_F32;
    p.weight_wide = aligned(a.weight, 16);
    p.x = a.x.data, p.x_row = a.x.row_stride, p.y = a.out.data, p.y_row = a.out.row_stride;
    p.weight = a.weight, p.bias = a.bias, p.state = a.state, p.state_slot = a.slot_stride, p.slots = a.slots;
    return launched(launch_conv_step(static_cast<dwp_dtype>(a.dtype), p, c.wide(a.channels, a.dtype), s));
}

// ---------------------------------------------------------------------------
// selective scan

// [groups, states] rows: checked as rows of their whole span.
void check_bc(Check &c, const dwp_rows &x, int64_t group_stride, int64_t t, int64_t batch, int64_t rows,
              int64_t groups, int64_t states) {
    c.require(groups == 1 || (group_stride >= states && group_stride <= kMaxStride));
    if (c.status != DWP_SUCCESS) return;
    const uintptr_t others = c.bits;
    c.bits = 0;
    c.rows(x, t, batch, rows, (groups - 1) * group_stride * (groups > 1) + states, false);
    c.bits_bc |= c.bits | uintptr_t(groups > 1 ? group_stride * size_of(t) : 0);
    c.bits = others;
}

bool scan_sizes_ok(int64_t dtype, int64_t softplus, int64_t channels, int64_t states, int64_t groups) {
    return dtype_ok(dtype) && (softplus == 0 || softplus == 1) && channels >= 1 && channels <= kMaxChannels &&
           states >= 1 && states <= kMaxStates && groups >= 1 && groups <= kMaxGroups && channels % groups == 0;
}

int64_t check_scan(Check &c, const dwp_selective_scan_args &a, bool backward) {
    c.require(scan_sizes_ok(a.dtype, a.softplus, a.channels, a.states, a.groups));
    const int64_t seqs = sequences(c, a.channels, a.batch, a.rows, a.num_segments, a.offsets);
    if (c.status != DWP_SUCCESS) return 0;
    const int64_t state = a.channels * a.states;
    const int64_t tiles = ceil_div(a.rows, DWP_SCAN_CHECKPOINT_ROWS);
    if (a.batch * a.rows > 0) {
        c.rows(a.u, a.dtype, a.batch, a.rows, a.channels, false);
        c.rows(a.dt, a.dtype, a.batch, a.rows, a.channels, false);
        if (a.z.data) c.rows(a.z, a.dtype, a.batch, a.rows, a.channels, false);
        check_bc(c, a.B, a.b_group_stride, a.dtype, a.batch, a.rows, a.groups, a.states);
        check_bc(c, a.C, a.c_group_stride, a.dtype, a.batch, a.rows, a.groups, a.states);
        if (!backward) c.rows(a.out, a.dtype, a.batch, a.rows, a.channels, true);
    }
    c.dense(a.A, DWP_F32, state, false, false, &c.bits_state);
    c.dense(a.D, DWP_F32, a.channels, false, true);
    c.dense(a.dt_bias, DWP_F32, a.channels, false, true);
    c.dense(a.initial_state, DWP_F32, seqs * state, false, true, &c.bits_state);
    if (!backward) c.dense(a.final_state, DWP_F32, seqs * state, true, true, &c.bits_state);
    c.dense(a.checkpoints, DWP_F32, a.batch * tiles * state, !backward, !backward, &c.bits_state);
    return seqs;
}

// Chunks of rows for the forward: as many as fill the GPU's warps once, where
// the channels alone fill less than half of them.  A cut costs a second walk
// over the rows, about 0.6 of the first; a warp alone on its scheduler runs at
// a third of the rate of three.  Measured at 8192 rows x 4096 channels x 16
// states (256 warps): 1 chunk 1013 us, 6 391, 7 293, 9 345, 14 309; at 65536 x
// 2048 (32 warps): 47 chunks 1311 us, 57 1086, 114 1107.
int64_t chunks_of(const dwp_selective_scan_args &a, int64_t units, int64_t slots) {
    if (2 * units >= slots) return 1;
    const int64_t most = ceil_div(a.rows, DWP_SCAN_CHECKPOINT_ROWS);
    return slots / units < most ? slots / units : most;
}

int64_t scan_units(const dwp_selective_scan_args &a, int64_t channels) {
    return a.batch * a.groups * ceil_div(a.channels / a.groups, channels);
}

// Whole tiles of rows to each chunk.
void set_chunks(ScanParams &p, int64_t chunks) {
    p.chunk_rows = ceil_div(p.tiles, chunks) * DWP_SCAN_CHECKPOINT_ROWS;
    p.chunks = ceil_div(p.rows, p.chunk_rows);
}

// Scratch of the states carried over chunks.
struct CarrySpace {
    size_t ends, sums, heads;
    explicit CarrySpace(const ScanParams &p)
        : ends(round16(size_t(p.batch * (p.chunks - 1) * p.channels * p.states) * 4u)),
          sums(round16(size_t(p.batch * (p.chunks - 1) * p.channels) * 4u)),
          heads(round16(size_t(p.batch * (p.chunks - 1)) * 4u)) {}
    size_t bytes() const { return ends + sums + heads; }
    void place(ScanParams &p, char *at) const {
        p.carry = reinterpret_cast<float *>(at);
        p.carry_sum = reinterpret_cast<float *>(at + ends);
        p.carry_head = reinterpret_cast<uint32_t *>(at + ends + sums);
    }
};

ScanParams scan_params(const dwp_selective_scan_args &a, uint32_t *segmap) {
    ScanParams p = {};
    p.channels = a.channels, p.groups = a.groups, p.group = a.channels / a.groups;
    p.batch = a.batch, p.rows = a.rows, p.states = int(a.states), p.softplus = int(a.softplus);
    p.tiles = ceil_div(a.rows, DWP_SCAN_CHECKPOINT_ROWS);
    p.chunks = 1, p.chunk_rows = p.tiles * DWP_SCAN_CHECKPOINT_ROWS;
    p.u = a.u.data, p.u_batch = a.u.batch_stride, p.u_row = a.u.row_stride;
    p.dt = a.dt.data, p.dt_batch = a.dt.batch_stride, p.dt_row = a.dt.row_stride;
    p.z = a.z.data, p.z_batch = a.z.batch_stride, p.z_row = a.z.row_stride;
    p.B = a.B.data, p.b_batch = a.B.batch_stride, p.b_row = a.B.row_stride, p.b_group = a.b_group_stride;
    p.C = a.C.data, p.c_batch = a.C.batch_stride, p.c_row = a.C.row_stride, p.c_group = a.c_group_stride;
    p.out = a.out.data, p.out_batch = a.out.batch_stride, p.out_row = a.out.row_stride;
    p.A = a.A, p.D = a.D, p.dt_bias = a.dt_bias, p.initial = a.initial_state;
    p.final = a.final_state, p.checkpoints = a.checkpoints;
    p.segmap = a.offsets ? segmap : nullptr;
    return p;
}

// How wide the scan's accesses may be.
void set_scan_access(ScanParams &p, const Check &c, const dwp_selective_scan_args &a) {
    const uintptr_t e = uintptr_t(size_of(a.dtype));
    p.wide = (c.bits & (2 * e - 1)) == 0 && p.group % 2 == 0 && (c.bits_bc & (4 * e - 1)) == 0 && a.states % 4 == 0;
    p.states_wide = (c.bits_state & 15u) == 0 && a.states % 4 == 0;
}

dwp_status scan_forward(const dwp_selective_scan_args &a, void *scratch, size_t *bytes, cudaStream_t s) {
    Check c;
    const int64_t seqs = check_scan(c, a, false);
    dwp_status st = c.status;
    if (st != DWP_SUCCESS) return st;
    ScanParams p = scan_params(a, static_cast<uint32_t *>(scratch));
    if (a.batch * a.rows > 0)
        set_chunks(p, chunks_of(a, scan_units(a, scan_warp_channels(a.states)), kSMs * kScanWarpsPerSM));
    const CarrySpace carry(p);
    const size_t map = a.offsets ? round16(size_t(a.rows) * 4u) : 0u;
    const size_t need = map + carry.bytes();
    if (!c.scratch(scratch, bytes, need, &st)) return st;
    const int64_t state = a.channels * a.states;
    if (a.final_state && (a.offsets || a.rows == 0)) {
        const cudaError_t err =
            launch_empty_states(DWP_F32, a.offsets, seqs, state, a.initial_state, a.final_state, s);
        if (err != cudaSuccess) return launched(err);
    }
    if (a.batch * a.rows == 0 || seqs == 0) return DWP_SUCCESS;
    if (a.offsets) {
        const cudaError_t err = launch_segment_map(a.offsets, uint32_t(seqs), uint32_t(a.rows),
                                                   static_cast<uint32_t *>(scratch), s);
        if (err != cudaSuccess) return launched(err);
    }
    carry.place(p, static_cast<char *>(scratch) + map);
    set_scan_access(p, c, a);
    return launched(launch_selscan(static_cast<dwp_dtype>(a.dtype), p, s));
}

dwp_status scan_backward(const dwp_selective_scan_backward_args &a, void *scratch, size_t *bytes, cudaStream_t s) {
    Check c;
    const dwp_selective_scan_args &f = a.scan;
    const int64_t seqs = check_scan(c, f, true);
    dwp_status st = c.status;
    if (st != DWP_SUCCESS) return st;
    const int64_t state = f.channels * f.states, n = f.batch * f.rows;
    if (n > 0) {
        c.rows(a.grad_out, f.dtype, f.batch, f.rows, f.channels, false);
        c.dense(a.grad_u, f.dtype, n * f.channels, true, false);
        c.dense(a.grad_dt, f.dtype, n * f.channels, true, false);
        c.require((a.grad_z != nullptr) == (f.z.data != nullptr));
        c.dense(a.grad_z, f.dtype, n * f.channels, true, true);
        c.dense(a.grad_B, f.dtype, n * f.groups * f.states, true, false);
        c.dense(a.grad_C, f.dtype, n * f.groups * f.states, true, false);
    }
    c.dense(a.grad_A, DWP_F32, state, true, false);
    c.dense(a.grad_D, DWP_F32, f.channels, true, true);
    c.dense(a.grad_dt_bias, DWP_F32, f.channels, true, true);
    c.dense(a.grad_final_state, DWP_F32, seqs * state, false, true, &c.bits_state);
    c.dense(a.grad_initial_state, DWP_F32, seqs * state, true, true);

    ScanBackwardParams p = {};
    p.f = scan_params(f, nullptr);
    const int64_t per = scan_block_channels(f.states), blocks = ceil_div(p.f.group, per);
    if (n > 0) set_chunks(p.f, chunks_of(f, scan_units(f, per), kSMs * kScanBackWarpsPerSM));
    const CarrySpace carry(p.f);
    const size_t map = f.offsets ? round16(size_t(f.rows) * 4u) : 0u;
    const size_t part = round16(size_t(f.batch * p.f.chunks * f.channels * (f.states + 2)) * 4u);
    const size_t bc = round16(size_t(blocks * n * f.groups * 2 * f.states) * 4u);
    if (!c.scratch(scratch, bytes, map + part + bc + carry.bytes(), &st)) return st;
    if (a.grad_initial_state && (f.offsets || f.rows == 0)) {
        const cudaError_t err = launch_empty_states(DWP_F32, f.offsets, seqs, state, a.grad_final_state,
                                                    a.grad_initial_state, s);
        if (err != cudaSuccess) return launched(err);
    }
    if (n == 0 || seqs == 0) {
        cudaError_t err = launch_clear(a.grad_A, size_t(state) * 4u, a.grad_D, size_t(f.channels) * 4u, s);
        if (err == cudaSuccess) err = launch_clear(a.grad_dt_bias, size_t(f.channels) * 4u, nullptr, 0, s);
        return launched(err);
    }
    char *at = static_cast<char *>(scratch);
    if (f.offsets) {
        p.f.segmap = reinterpret_cast<uint32_t *>(at);
        const cudaError_t err = launch_segment_map(f.offsets, uint32_t(seqs), uint32_t(f.rows),
                                                   reinterpret_cast<uint32_t *>(at), s);
        if (err != cudaSuccess) return launched(err);
    }
    p.partial = reinterpret_cast<float *>(at + map);
    p.partial_bc = reinterpret_cast<float *>(at + map + part);
    p.grad_out = a.grad_out.data, p.grad_batch = a.grad_out.batch_stride, p.grad_row = a.grad_out.row_stride;
    p.grad_final = a.grad_final_state, p.grad_initial = a.grad_initial_state;
    p.grad_u = a.grad_u, p.grad_dt = a.grad_dt, p.grad_z = a.grad_z, p.grad_B = a.grad_B, p.grad_C = a.grad_C;
    set_scan_access(p.f, c, f);
    carry.place(p.f, at + map + part + bc);
    const auto t = static_cast<dwp_dtype>(f.dtype);
    if (p.f.chunks > 1) {
        ScanParams r = p.f;  // as the walk back reads it
        r.u = p.grad_out, r.u_batch = p.grad_batch, r.u_row = p.grad_row;
        r.B = p.f.C, r.b_batch = p.f.c_batch, r.b_row = p.f.c_row, r.b_group = p.f.c_group;
        r.initial = p.grad_final;
        const cudaError_t err = launch_scan_walk_back(t, r, s);
        if (err != cudaSuccess) return launched(err);
    }
    cudaError_t err = launch_selscan_backward(t, p, s);
    if (err != cudaSuccess) return launched(err);
    const ColumnOut o{{a.grad_A, a.grad_D, a.grad_dt_bias},
                      {state, state + f.channels, state + 2 * f.channels},
                      1};
    return launched(launch_column_sums(p.partial, f.batch * p.f.chunks, state + 2 * f.channels, o, s));
}

dwp_status scan_step(const dwp_selective_scan_step_args &a, cudaStream_t s) {
    Check c;
    c.require(scan_sizes_ok(a.dtype, a.softplus, a.channels, a.states, a.groups) && a.batch >= 0 &&
              a.batch <= kMaxRows);
    if (c.status != DWP_SUCCESS) return c.status;
    if (a.batch == 0) return DWP_SUCCESS;
    c.rows(a.u, a.dtype, 1, a.batch, a.channels, false);
    c.rows(a.dt, a.dtype, 1, a.batch, a.channels, false);
    if (a.z.data) c.rows(a.z, a.dtype, 1, a.batch, a.channels, false);
    check_bc(c, a.B, a.b_group_stride, a.dtype, 1, a.batch, a.groups, a.states);
    check_bc(c, a.C, a.c_group_stride, a.dtype, 1, a.batch, a.groups, a.states);
    c.rows(a.out, a.dtype, 1, a.batch, a.channels, true);
    c.dense(a.A, DWP_F32, a.channels * a.states, false, false, &c.bits_state);
    c.bits_state |= reinterpret_cast<uintptr_t>(a.state);
    c.dense(a.D, DWP_F32, a.channels, false, true);
    c.dense(a.dt_bias, DWP_F32, a.channels, false, true);
    check_slots(c, a.state, DWP_F32, a.batch, a.num_slots, a.slot_stride, a.channels * a.states, a.slots);
    if (c.status != DWP_SUCCESS) return c.status;
    if (c.regions.clash()) return DWP_ERR_ALIASING;
    ScanStepParams p = {};
    p.channels = a.channels, p.groups = a.groups, p.group = a.channels / a.groups;
    p.batch = a.batch, p.num_slots = a.num_slots, p.states = int(a.states), p.softplus = int(a.softplus);
    p.u = a.u.data, p.u_row = a.u.row_stride, p.dt = a.dt.data, p.dt_row = a.dt.row_stride;
    p.z = a.z.data, p.z_row = a.z.row_stride, p.out = a.out.data, p.out_row = a.out.row_stride;
    p.B = a.B.data, p.b_row = a.B.row_stride, p.b_group = a.b_group_stride;
    p.C = a.C.data, p.c_row = a.C.row_stride, p.c_group = a.c_group_stride;
    p.A = a.A, p.D = a.D, p.dt_bias = a.dt_bias;
    p.state = a.state, p.state_slot = a.slot_stride, p.slots = a.slots;
    const uintptr_t e = uintptr_t(size_of(a.dtype));
    p.wide = a.states % 4 == 0 && (c.bits_bc & (4 * e - 1)) == 0 &&
             ((c.bits_state | uintptr_t(a.slot_stride * 4)) & 15u) == 0;
    return launched(launch_selscan_step(static_cast<dwp_dtype>(a.dtype), p, s));
}

// ---------------------------------------------------------------------------
// block norm

void check_norm(Check &c, const dwp_norm_args &a) {
    c.require(dtype_ok(a.dtype) && (a.weight_dtype == a.dtype || a.weight_dtype == DWP_F32) &&
              (a.residual_dtype == a.dtype || a.residual_dtype == DWP_F32) &&
              (a.gate_after == 0 || a.gate_after == 1) && a.channels >= 1 && a.channels <= kMaxChannels &&
              a.groups >= 1 && a.groups <= kMaxGroups && a.channels % a.groups == 0 &&
              a.channels / a.groups <= DWP_NORM_MAX_GROUP && a.rows >= 0 && a.rows <= kMaxRows &&
              a.rows * a.groups <= kMaxRows && a.eps >= 0.0);
    if (c.status != DWP_SUCCESS) return;
    c.dense(a.weight, a.weight_dtype, a.channels, false, false, &c.bits);
    c.dense(a.scale, a.weight_dtype, a.channels, false, true, &c.bits);
}

NormParams norm_params(const dwp_norm_args &a) {
    NormParams p = {};
    p.channels = a.channels, p.groups = a.groups, p.group = a.channels / a.groups, p.rows = a.rows;
    p.eps = float(a.eps), p.gate_after = int(a.gate_after);
    p.weight_f32 = a.weight_dtype == DWP_F32, p.residual_f32 = a.residual_dtype == DWP_F32;
    p.x = a.x.data, p.x_row = a.x.row_stride, p.residual = a.residual.data, p.residual_row = a.residual.row_stride;
    p.gate = a.gate.data, p.gate_row = a.gate.row_stride, p.sum = a.sum.data, p.sum_row = a.sum.row_stride;
    p.y = a.out.data, p.y_row = a.out.row_stride, p.weight = a.weight, p.scale = a.scale;
    return p;
}

bool same_rows(const dwp_rows &a, const dwp_rows &b) { return a.data == b.data && a.row_stride == b.row_stride; }

dwp_status norm_forward(const dwp_norm_args &a, cudaStream_t s) {
    Check c;
    check_norm(c, a);
    if (c.status != DWP_SUCCESS) return c.status;
    if (a.rows == 0) return DWP_SUCCESS;  // no data, and maybe no addresses
    c.require((a.residual.data != nullptr) == (a.sum.data != nullptr) && (!a.scale || a.residual.data));
    // an output that is its input exactly counts once, as the output
    c.rows(a.x, a.dtype, 1, a.rows, a.channels, false, !same_rows(a.x, a.out));
    if (a.residual.data) {
        c.rows(a.residual, a.residual_dtype, 1, a.rows, a.channels, false, !same_rows(a.residual, a.sum));
        c.rows(a.sum, a.residual_dtype, 1, a.rows, a.channels, true);
    }
    if (a.gate.data) c.rows(a.gate, a.dtype, 1, a.rows, a.channels, false);
    c.rows(a.out, a.dtype, 1, a.rows, a.channels, true);
    if (c.status != DWP_SUCCESS) return c.status;
    if (c.regions.clash()) return DWP_ERR_ALIASING;
    return launched(launch_norm(static_cast<dwp_dtype>(a.dtype), norm_params(a), c.wide(a.channels / a.groups, a.dtype), s));
}

// Blocks that share a group's rows in the gradient: those that run at once
// (512 threads of 128 registers fill an SM), so that none waits for another's
// end.  Gated norm of 4096 x 8192 f16 in 8 groups: 512 threads an SM 97 us,
// 768 122, 1024 102.
int64_t norm_blocks(const dwp_norm_args &a, bool wide) {
    const int64_t threads = norm_backward_threads(static_cast<dwp_dtype>(a.dtype), a.channels / a.groups, wide);
    int64_t blocks = kSMs * (512 / threads) / a.groups;
    if (8 * blocks > a.rows) blocks = ceil_div(a.rows, 8);  // eight rows or more to each
    return blocks < 1 && a.rows > 0 ? 1 : blocks;
}

dwp_status norm_backward(const dwp_norm_backward_args &a, void *scratch, size_t *bytes, cudaStream_t s) {
    Check c;
    const dwp_norm_args &f = a.norm;
    check_norm(c, f);
    dwp_status st = c.status;
    if (st != DWP_SUCCESS) return st;
    const bool resid = f.sum.data != nullptr;
    c.require((a.grad_scale != nullptr) == (f.scale != nullptr));
    if (f.rows > 0) {
        c.require((!f.scale || resid) && (resid || (!a.grad_residual.data && !a.grad_sum.data)) &&
                  (a.grad_gate.data != nullptr) == (f.gate.data != nullptr));
        if (resid) c.rows(f.sum, f.residual_dtype, 1, f.rows, f.channels, false);
        if (!resid || f.scale) c.rows(f.x, f.dtype, 1, f.rows, f.channels, false);
        if (f.gate.data) c.rows(f.gate, f.dtype, 1, f.rows, f.channels, false);
        c.rows(a.grad_out, f.dtype, 1, f.rows, f.channels, false);
        if (a.grad_sum.data) c.rows(a.grad_sum, f.residual_dtype, 1, f.rows, f.channels, false);
        if (a.grad_x.data) c.rows(a.grad_x, f.dtype, 1, f.rows, f.channels, true);
        if (a.grad_residual.data) c.rows(a.grad_residual, f.residual_dtype, 1, f.rows, f.channels, true);
        if (f.gate.data) c.rows(a.grad_gate, f.dtype, 1, f.rows, f.channels, true);
    }
    c.dense(a.grad_weight, DWP_F32, f.channels, true, false);
    c.dense(a.grad_scale, DWP_F32, f.channels, true, true);
    const int64_t blocks = norm_blocks(f, c.wide(f.channels / f.groups, f.dtype));
    const int64_t planes = f.scale ? 2 : 1;
    const size_t need = round16(size_t(blocks * planes * f.channels) * 4u);
    if (!c.scratch(scratch, bytes, need, &st)) return st;
    if (f.rows == 0)
        return launched(launch_clear(a.grad_weight, size_t(f.channels) * 4u, a.grad_scale, size_t(f.channels) * 4u, s));
    NormBackwardParams p = {};
    p.n = norm_params(f);
    p.blocks = blocks;
    p.v = resid ? f.sum.data : f.x.data, p.v_row = resid ? f.sum.row_stride : f.x.row_stride;
    p.v_f32 = resid ? f.residual_dtype == DWP_F32 : f.dtype == DWP_F32;
    p.x_in = f.scale ? f.x.data : nullptr, p.xin_row = f.x.row_stride;
    p.grad_out = a.grad_out.data, p.grad_row = a.grad_out.row_stride;
    p.grad_sum = a.grad_sum.data, p.gsum_row = a.grad_sum.row_stride;
    p.grad_x = a.grad_x.data, p.gx_row = a.grad_x.row_stride;
    p.grad_residual = a.grad_residual.data, p.gres_row = a.grad_residual.row_stride;
    p.grad_gate = a.grad_gate.data, p.ggate_row = a.grad_gate.row_stride;
    p.partial = static_cast<float *>(scratch);
    cudaError_t err = launch_norm_backward(static_cast<dwp_dtype>(f.dtype), p, c.wide(f.channels / f.groups, f.dtype), s);
    if (err != cudaSuccess) return launched(err);
    const ColumnOut o{{a.grad_weight, a.grad_scale, nullptr}, {f.channels, planes * f.channels, 0}, 1};
    return launched(launch_column_sums(p.partial, blocks, planes * f.channels, o, s));
}

// ---------------------------------------------------------------------------
// layer norm

void check_layer_norm(Check &c, const dwp_layer_norm_args &a) {
    c.require(dtype_ok(a.dtype) && (a.weight_dtype == a.dtype || a.weight_dtype == DWP_F32) &&
              (a.residual_dtype == a.dtype || a.residual_dtype == DWP_F32) && a.channels >= 1 &&
              a.channels <= kMaxChannels && a.groups >= 1 && a.groups <= kMaxGroups && a.channels % a.groups == 0 &&
              a.channels / a.groups <= DWP_NORM_MAX_GROUP && a.rows >= 0 && a.rows <= kMaxRows &&
              a.rows * a.groups <= kMaxRows && a.eps >= 0.0);
    if (c.status != DWP_SUCCESS) return;
    c.dense(a.weight, a.weight_dtype, a.channels, false, true, &c.bits);
    c.dense(a.bias, a.weight_dtype, a.channels, false, true, &c.bits);
}

LayerNormParams layer_norm_params(const dwp_layer_norm_args &a) {
    LayerNormParams p = {};
    p.channels = a.channels, p.groups = a.groups, p.group = a.channels / a.groups, p.rows = a.rows;
    p.eps = float(a.eps), p.weight_f32 = a.weight_dtype == DWP_F32, p.residual_f32 = a.residual_dtype == DWP_F32;
    p.x = a.x.data, p.x_row = a.x.row_stride, p.residual = a.residual.data, p.residual_row = a.residual.row_stride;
    p.sum = a.sum.data, p.sum_row = a.sum.row_stride, p.y = a.out.data, p.y_row = a.out.row_stride;
    p.weight = a.weight, p.bias = a.bias;
    return p;
}

dwp_status layer_norm_forward(const dwp_layer_norm_args &a, cudaStream_t s) {
    Check c;
    check_layer_norm(c, a);
    if (c.status != DWP_SUCCESS) return c.status;
    if (a.rows == 0) return DWP_SUCCESS;  // no data, and maybe no addresses
    c.require((a.residual.data != nullptr) == (a.sum.data != nullptr));
    // an output that is its input exactly counts once, as the output
    c.rows(a.x, a.dtype, 1, a.rows, a.channels, false, !same_rows(a.x, a.out));
    if (a.residual.data) {
        c.rows(a.residual, a.residual_dtype, 1, a.rows, a.channels, false, !same_rows(a.residual, a.sum));
        c.rows(a.sum, a.residual_dtype, 1, a.rows, a.channels, true);
    }
    c.rows(a.out, a.dtype, 1, a.rows, a.channels, true);
    if (c.status != DWP_SUCCESS) return c.status;
    if (c.regions.clash()) return DWP_ERR_ALIASING;
    return launched(launch_layer_norm(static_cast<dwp_dtype>(a.dtype), layer_norm_params(a),
                                      c.wide(a.channels / a.groups, a.dtype), s));
}

// Blocks that share a group's rows in the gradient: those that run at once, each
// team with four rows or more.
int64_t layer_norm_blocks(const dwp_layer_norm_args &a, bool wide) {
    int64_t per_sm;
    const int64_t teams = layer_norm_teams(static_cast<dwp_dtype>(a.dtype), a.channels / a.groups, wide, per_sm);
    int64_t blocks = kSMs * per_sm / a.groups;
    if (4 * blocks * teams > a.rows) blocks = ceil_div(a.rows, 4 * teams);
    return blocks < 1 && a.rows > 0 ? 1 : blocks;
}

dwp_status layer_norm_backward(const dwp_layer_norm_backward_args &a, void *scratch, size_t *bytes, cudaStream_t s) {
    Check c;
    const dwp_layer_norm_args &f = a.norm;
    check_layer_norm(c, f);
    dwp_status st = c.status;
    if (st != DWP_SUCCESS) return st;
    const bool resid = f.sum.data != nullptr;
    if (f.rows > 0) {
        c.require(resid || (!a.grad_residual.data && !a.grad_sum.data && f.residual_dtype == f.dtype));
        if (resid) c.rows(f.sum, f.residual_dtype, 1, f.rows, f.channels, false);
        else c.rows(f.x, f.dtype, 1, f.rows, f.channels, false);
        c.rows(a.grad_out, f.dtype, 1, f.rows, f.channels, false);
        if (a.grad_sum.data) c.rows(a.grad_sum, f.residual_dtype, 1, f.rows, f.channels, false);
        if (a.grad_x.data) c.rows(a.grad_x, f.dtype, 1, f.rows, f.channels, true);
        if (a.grad_residual.data) c.rows(a.grad_residual, f.residual_dtype, 1, f.rows, f.channels, true);
    }
    c.dense(a.grad_weight, DWP_F32, f.channels, true, true);
    c.dense(a.grad_bias, DWP_F32, f.channels, true, true);
    const bool wide = c.wide(f.channels / f.groups, f.dtype), sums = a.grad_weight || a.grad_bias;
    const int64_t blocks = layer_norm_blocks(f, wide);
    if (!c.scratch(scratch, bytes, sums ? round16(size_t(blocks * 2 * f.channels) * 4u) : 0u, &st)) return st;
    if (f.rows == 0)
        return launched(launch_clear(a.grad_weight, size_t(f.channels) * 4u, a.grad_bias, size_t(f.channels) * 4u, s));
    LayerNormBackwardParams p = {};
    p.n = layer_norm_params(f);
    p.blocks = blocks;
    p.v = resid ? f.sum.data : f.x.data, p.v_row = resid ? f.sum.row_stride : f.x.row_stride;
    p.v_f32 = resid ? f.residual_dtype == DWP_F32 : f.dtype == DWP_F32;
    p.grad_out = a.grad_out.data, p.grad_row = a.grad_out.row_stride;
    p.grad_sum = a.grad_sum.data, p.gsum_row = a.grad_sum.row_stride;
    p.grad_x = a.grad_x.data, p.gx_row = a.grad_x.row_stride;
    p.grad_residual = a.grad_residual.data, p.gres_row = a.grad_residual.row_stride;
    p.partial = sums ? static_cast<float *>(scratch) : nullptr;
    const cudaError_t err = launch_layer_norm_backward(static_cast<dwp_dtype>(f.dtype), p, wide, s);
    if (err != cudaSuccess || !sums) return launched(err);
    const ColumnOut o{{a.grad_weight, a.grad_bias, nullptr}, {f.channels, 2 * f.channels, 0}, 1};
    return launched(launch_column_sums(p.partial, blocks, 2 * f.channels, o, s));
}

}  // namespace

extern "C" {

dwp_status dwp_causal_conv(const dwp_conv_args *args, dwp_stream stream) {
    if (!args) return DWP_ERR_INVALID_VALUE;
    return conv_forward(*args, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_causal_conv_backward(const dwp_conv_backward_args *args, void *d_scratch, size_t *scratch_bytes,
                                    dwp_stream stream) {
    if (!args || !scratch_bytes) return DWP_ERR_INVALID_VALUE;
    return conv_backward(*args, d_scratch, scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_causal_conv_step(const dwp_conv_step_args *args, dwp_stream stream) {
    if (!args) return DWP_ERR_INVALID_VALUE;
    return conv_step(*args, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_selective_scan(const dwp_selective_scan_args *args, void *d_scratch, size_t *scratch_bytes,
                              dwp_stream stream) {
    if (!args || !scratch_bytes) return DWP_ERR_INVALID_VALUE;
    return scan_forward(*args, d_scratch, scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_selective_scan_backward(const dwp_selective_scan_backward_args *args, void *d_scratch,
                                       size_t *scratch_bytes, dwp_stream stream) {
    if (!args || !scratch_bytes) return DWP_ERR_INVALID_VALUE;
    return scan_backward(*args, d_scratch, scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_selective_scan_step(const dwp_selective_scan_step_args *args, dwp_stream stream) {
    if (!args) return DWP_ERR_INVALID_VALUE;
    return scan_step(*args, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_block_norm(const dwp_norm_args *args, dwp_stream stream) {
    if (!args) return DWP_ERR_INVALID_VALUE;
    return norm_forward(*args, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_block_norm_backward(const dwp_norm_backward_args *args, void *d_scratch, size_t *scratch_bytes,
                                   dwp_stream stream) {
    if (!args || !scratch_bytes) return DWP_ERR_INVALID_VALUE;
    return norm_backward(*args, d_scratch, scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_layer_norm(const dwp_layer_norm_args *args, dwp_stream stream) {
    if (!args) return DWP_ERR_INVALID_VALUE;
    return layer_norm_forward(*args, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_layer_norm_backward(const dwp_layer_norm_backward_args *args, void *d_scratch, size_t *scratch_bytes,
                                   dwp_stream stream) {
    if (!args || !scratch_bytes) return DWP_ERR_INVALID_VALUE;
    return layer_norm_backward(*args, d_scratch, scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
