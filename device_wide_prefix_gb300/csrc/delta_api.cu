// C entry points of the gated delta rule: argument validation, the scratch
// size query and the launches.  Validation happens before any CUDA call.
#include "sequence_check.h"

namespace {

using namespace dwp;

constexpr int64_t kMaxHeadSize = 128;
constexpr int64_t kTile = int64_t(DWP_DELTA_CHUNK) * DWP_DELTA_CHUNK;

bool delta_sizes_ok(int64_t dtype, int64_t beta_dtype, int64_t keys, int64_t values, int64_t key_heads, int64_t heads,
                    double scale) {
    return dtype_ok(dtype) && (beta_dtype == dtype || beta_dtype == DWP_F32) && keys >= 1 && keys <= kMaxHeadSize &&
           values >= 1 && values <= kMaxHeadSize && key_heads >= 1 && heads >= key_heads && heads <= kMaxGroups &&
           heads % key_heads == 0 && float(scale) - float(scale) == 0.0f;  // finite as the kernels take it
}

DeltaRows delta_rows(const dwp_heads &x) {
    return {static_cast<char *>(x.data), x.batch_stride, x.row_stride, x.head_stride};
}
DeltaRows delta_rows(const dwp_rows &x) { return {static_cast<char *>(x.data), x.batch_stride, x.row_stride, 1}; }
// Dense [batch, rows, heads, inner].
DeltaRows delta_dense(void *p, int64_t rows, int64_t heads, int64_t inner) {
    return {static_cast<char *>(p), rows * heads * inner, heads * inner, inner};
}

// Chunk places of a call: of each batch entry, or of the packed rows, where a
// segment's last chunk may be short.
int64_t delta_chunks(const dwp_delta_args &a) { return ceil_div(a.rows, DWP_DELTA_CHUNK); }
int64_t delta_slots(const dwp_delta_args &a) {
    return a.offsets ? a.rows / DWP_DELTA_CHUNK + a.num_segments : a.batch * delta_chunks(a);
}

// Words of a kept state, keys in whole tiles, and of a chunk's kept rows, values in whole tiles.
int64_t delta_state(const dwp_delta_args &a) { return ceil_div(a.keys, 64) * 64 * a.values; }
int64_t delta_kept_rows(const dwp_delta_args &a) { return DWP_DELTA_CHUNK * ceil_div(a.values, 64) * 64; }
// Whether rows with these address and stride bits are whole 16-byte pieces.
bool delta_wide(uintptr_t bits, const dwp_delta_args &a) {
    return ((bits | uintptr_t((a.keys | a.values) * size_of(a.dtype))) & 15u) == 0;
}

// Parts that a call's sequences are cut in, and the words that takes (of bf16;
// wherever its rows lie, so that a size does not go by addresses).
int64_t delta_parts_of(const dwp_delta_args &a, int64_t seqs) {
    return a.offsets || a.dtype != DWP_BF16 ? 1 : delta_parts(seqs * a.heads, delta_chunks(a));
}
size_t delta_part_bytes(const dwp_delta_args &a, int64_t seqs) {
    const int64_t parts = delta_parts_of(a, seqs);
    return parts == 1 ? 0u : round16(size_t(seqs * parts * a.heads * (2 * a.keys * a.values + a.keys * a.keys)) * 4u);
}
void set_parts(DeltaParams &p, const dwp_delta_args &a, int64_t seqs, bool maps, void *at) {
    // only rows that come by maps are cut
    p.parts = maps ? delta_parts_of(a, seqs) : 1, p.part_chunks = ceil_div(p.chunks, p.parts);
    const int64_t places = seqs * p.parts * a.heads;
    p.part_starts = static_cast<float *>(at);
    p.part_ends = p.part_starts + places * a.keys * a.values;
    p.part_maps = p.part_ends + places * a.keys * a.values;
}

int64_t check_delta(Check &c, const dwp_delta_args &a, bool backward, uintptr_t &out_bits) {
    c.require(delta_sizes_ok(a.dtype, a.beta_dtype, a.keys, a.values, a.key_heads, a.heads, a.scale));
    const int64_t seqs = sequences(c, 1, a.batch, a.rows, a.num_segments, a.offsets);
    if (c.status != DWP_SUCCESS) return 0;
    const int64_t state = a.heads * a.keys * a.values;
    if (a.batch * a.rows > 0) {
        c.heads(a.q, a.dtype, a.batch, a.rows, a.key_heads, a.keys, false);
        c.heads(a.k, a.dtype, a.batch, a.rows, a.key_heads, a.keys, false);
        c.heads(a.v, a.dtype, a.batch, a.rows, a.heads, a.values, false);
        const uintptr_t others = c.bits;
        c.bits = 0;
        if (!backward) c.heads(a.out, a.dtype, a.batch, a.rows, a.heads, a.values, true);
        out_bits = c.bits;
        if (a.g.data) c.rows(a.g, DWP_F32, a.batch, a.rows, a.heads, false);
        c.rows(a.beta, a.beta_dtype, a.batch, a.rows, a.heads, false);
        c.bits = others;
    }
    c.dense(a.initial_state, DWP_F32, seqs * state, false, true);
    if (!backward) c.dense(a.final_state, DWP_F32, seqs * state, true, true);
    if (c.status != DWP_SUCCESS) return seqs;
    const int64_t each = delta_kept_rows(a) + delta_state(a) + 2 * kTile;
    c.dense(a.checkpoints, DWP_F32, delta_slots(a) * a.heads * each, !backward, !backward);
    if (!aligned(a.checkpoints, 16)) c.fail(DWP_ERR_MISALIGNED);
    return seqs;
}

DeltaParams delta_params(const dwp_delta_args &a, int64_t seqs, void *scratch) {
    DeltaParams p = {};
    p.keys = int(a.keys), p.values = int(a.values), p.key_heads = int(a.key_heads), p.heads = int(a.heads);
    p.batch = a.batch, p.rows = a.rows, p.sequences = seqs, p.chunks = delta_chunks(a), p.slots = delta_slots(a);
    p.scale = float(a.scale), p.beta_f32 = a.beta_dtype == DWP_F32;
    p.q = delta_rows(a.q), p.k = delta_rows(a.k), p.v = delta_rows(a.v), p.out = delta_rows(a.out);
    p.g = delta_rows(a.g), p.beta = delta_rows(a.beta);
    p.offsets = a.offsets, p.initial = a.initial_state, p.final = a.final_state;
#ifdef DWP_DELTA_TEST
    delta_stall(p);
#endif
    const int64_t places = p.slots * a.heads;
    p.inverse = a.checkpoints ? a.checkpoints : static_cast<float *>(scratch);
    p.weights = p.inverse + places * kTile;
    if (a.checkpoints) {
        p.u = p.weights + places * kTile;
        p.states = p.u + places * delta_kept_rows(a);
    }
    return p;
}

dwp_status delta_forward(const dwp_delta_args &a, void *scratch, size_t *bytes, cudaStream_t s) {
    Check c;
    uintptr_t out_bits = 0;
    const int64_t seqs = check_delta(c, a, false, out_bits);
    dwp_status st = c.status;
    if (st != DWP_SUCCESS) return st;
    const size_t need = a.checkpoints ? 0u : size_t(delta_slots(a) * a.heads * 2 * kTile) * 4u;
    if (!c.scratch(scratch, bytes, need + delta_part_bytes(a, seqs), &st)) return st;
    if (seqs == 0) return DWP_SUCCESS;
    DeltaParams p = delta_params(a, seqs, scratch);
    p.wide = delta_wide(c.bits, a);
    p.out_wide = delta_wide(out_bits, a);
    const auto t = static_cast<dwp_dtype>(a.dtype);
    const DeltaMaps maps = delta_maps(t, p, nullptr);
    set_parts(p, a, seqs, maps.made, static_cast<char *>(scratch) + need);
    if (a.batch * a.rows > 0) {
        const cudaError_t err = launch_delta_local(t, p, maps, s);
        if (err != cudaSuccess) return launched(err);
    } else if (!a.final_state) {
        return DWP_SUCCESS;
    }
    return launched(launch_delta_chain(t, p, maps, s));
}

dwp_status delta_backward(const dwp_delta_backward_args &a, void *scratch, size_t *bytes, cudaStream_t s) {
    Check c;
    const dwp_delta_args &f = a.delta;
    uintptr_t out_bits = 0;
    const int64_t seqs = check_delta(c, f, true, out_bits);
    dwp_status st = c.status;
    if (st != DWP_SUCCESS) return st;
    const int64_t n = f.batch * f.rows, state = f.heads * f.keys * f.values;
    bool wide = false;
    if (n > 0) {
        c.heads(a.grad_out, f.dtype, f.batch, f.rows, f.heads, f.values, false);
        wide = delta_wide(c.bits, f);
        c.dense(a.grad_q, f.dtype, n * f.key_heads * f.keys, true, false);
        c.dense(a.grad_k, f.dtype, n * f.key_heads * f.keys, true, false);
        c.dense(a.grad_v, f.dtype, n * f.heads * f.values, true, false);
        c.require(!a.grad_g || f.g.data);
        c.dense(a.grad_g, DWP_F32, n * f.heads, true, true);
        c.dense(a.grad_beta, f.beta_dtype, n * f.heads, true, false);
    }
    c.dense(a.grad_final_state, DWP_F32, seqs * state, false, true);
    c.dense(a.grad_initial_state, DWP_F32, seqs * state, true, true);
    const int64_t places = delta_slots(f) * f.heads;
    const size_t dr = size_t(places * delta_kept_rows(f)) * 4u;
    const size_t ends = round16(size_t(places * delta_state(f)) * 4u);
    if (!c.scratch(scratch, bytes, dr + ends + delta_part_bytes(f, seqs), &st)) return st;
    if (seqs == 0) return DWP_SUCCESS;
    DeltaBackwardParams p = {};
    p.f = delta_params(f, seqs, nullptr);
    p.f.wide = wide;
    p.grad_out = delta_rows(a.grad_out);
    p.grad_q = delta_dense(a.grad_q, f.rows, f.key_heads, f.keys);
    p.grad_k = delta_dense(a.grad_k, f.rows, f.key_heads, f.keys);
    p.grad_v = delta_dense(a.grad_v, f.rows, f.heads, f.values);
    p.grad_g = delta_dense(a.grad_g, f.rows, f.heads, 1);
    p.grad_beta = delta_dense(a.grad_beta, f.rows, f.heads, 1);
    p.grad_final = a.grad_final_state, p.grad_initial = a.grad_initial_state;
    char *at = static_cast<char *>(scratch);
    p.dr = reinterpret_cast<float *>(at);
    p.ends = reinterpret_cast<float *>(at + dr);
    p.wide = aligned(a.grad_v, 16);
    const auto t = static_cast<dwp_dtype>(f.dtype);
    const DeltaMaps maps = delta_maps(t, p.f, &p.grad_out);
    set_parts(p.f, f, seqs, maps.made, at + dr + ends);
    if (n > 0 || a.grad_initial_state) {
        const cudaError_t err = launch_delta_chain_back(t, p, maps, s);
        if (err != cudaSuccess) return launched(err);
    }
    return n > 0 ? launched(launch_delta_grad(t, p, maps, s)) : DWP_SUCCESS;
}

dwp_status delta_step(const dwp_delta_step_args &a, cudaStream_t s) {
    Check c;
    c.require(delta_sizes_ok(a.dtype, a.beta_dtype, a.keys, a.values, a.key_heads, a.heads, a.scale) && a.batch >= 0 &&
              a.batch <= kMaxRows);
    if (c.status != DWP_SUCCESS) return c.status;
    if (a.batch == 0) return DWP_SUCCESS;
    c.heads(a.q, a.dtype, 1, a.batch, a.key_heads, a.keys, false);
    c.heads(a.k, a.dtype, 1, a.batch, a.key_heads, a.keys, false);
    if (a.g.data) c.rows(a.g, DWP_F32, 1, a.batch, a.heads, false);
    c.rows(a.beta, a.beta_dtype, 1, a.batch, a.heads, false);
    c.bits = 0;
    c.heads(a.v, a.dtype, 1, a.batch, a.heads, a.values, false);
    c.heads(a.out, a.dtype, 1, a.batch, a.heads, a.values, true);
    const uintptr_t bits = c.bits;
    c.bits = 0;
    check_slots(c, a.state, DWP_F32, a.batch, a.num_slots, a.slot_stride, a.heads * a.keys * a.values, a.slots);
    if (c.status != DWP_SUCCESS) return c.status;
    if (c.regions.clash()) return DWP_ERR_ALIASING;
    DeltaStepParams p = {};
    p.keys = int(a.keys), p.values = int(a.values), p.key_heads = int(a.key_heads), p.heads = int(a.heads);
    p.batch = a.batch, p.num_slots = a.num_slots, p.scale = float(a.scale), p.beta_f32 = a.beta_dtype == DWP_F32;
    p.q = delta_rows(a.q), p.k = delta_rows(a.k), p.v = delta_rows(a.v), p.out = delta_rows(a.out);
    p.g = delta_rows(a.g), p.beta = delta_rows(a.beta);
    p.state = a.state, p.state_slot = a.slot_stride, p.slots = a.slots;
    p.wide = a.values % 4 == 0 && (bits & uintptr_t(4 * size_of(a.dtype) - 1)) == 0 && (c.bits & 15u) == 0;
    return launched(launch_delta_step(static_cast<dwp_dtype>(a.dtype), p, s));
}

}  // namespace

extern "C" {

dwp_status dwp_gated_delta_rule(const dwp_delta_args *args, void *d_scratch, size_t *scratch_bytes, dwp_stream stream) {
    if (!args || !scratch_bytes) return DWP_ERR_INVALID_VALUE;
    return delta_forward(*args, d_scratch, scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_gated_delta_rule_backward(const dwp_delta_backward_args *args, void *d_scratch, size_t *scratch_bytes,
                                         dwp_stream stream) {
    if (!args || !scratch_bytes) return DWP_ERR_INVALID_VALUE;
    return delta_backward(*args, d_scratch, scratch_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dwp_status dwp_gated_delta_rule_step(const dwp_delta_step_args *args, dwp_stream stream) {
    if (!args) return DWP_ERR_INVALID_VALUE;
    return delta_step(*args, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
