// The gated delta rule: what its kernels share.
//
// Per sequence and head, with a state S of keys x values and a = exp(g):
//
//   S' = a S;  u = beta (v - S'^T k);  S = S' + k u^T;  o = scale S^T q
//
// Over a chunk of 64 rows that begins at state S0, with G the running sum of
// g in the chunk (G_C its last) and M_ij = exp(G_i - G_j) k_i.k_j:
//
//   T = (1 + strictly lower part of diag(beta) M)^-1
//   U = T diag(beta) (V - diag(e^G) K S0)
//   O = scale (diag(e^G) Q S0 + A U),   A_ij = exp(G_i - G_j) q_i.k_j, j <= i
//   S1 = e^{G_C} S0 + K^T diag(e^{G_C - G}) U
//
// T and A depend on the chunk alone (delta_local.cu, all chunks at once); the
// states go from chunk to chunk (delta_chain.cuh).  The gradient walks the
// chunks back for the states' gradients (delta_chain.cuh) and then has all
// chunks at once again (delta_grad.cuh).
#pragma once

#include "sequence.cuh"
#include "tensor.cuh"

namespace dwp {

constexpr int kChunk = 64;

// Log decays below this count as this: its exponential is 0 in f32 all the
// same, and sums of it stay finite, so that differences of sums are numbers.
constexpr float kLeastDecay = -110.0f;

// One chunk: its rows, and the sequence it belongs to.
struct DeltaChunk {
    int64_t batch, row;  // batch entry and first row in it
    int rows;            // rows in it, 0: no chunk here
    int64_t seq;
};

// First row and rows of a sequence, for any offsets inside the rows.
__device__ __forceinline__ void delta_sequence(const DeltaParams &p, int64_t seq, int64_t &batch, int64_t &row,
                                               int64_t &rows, int64_t &slot) {
    if (p.offsets) {
        const int64_t lo = min(int64_t(p.offsets[seq]), p.rows), hi = min(int64_t(p.offsets[seq + 1]), p.rows);
        batch = 0, row = lo, rows = hi > lo ? hi - lo : 0;
        slot = lo / kChunk + seq;  // sequences' places are apart: ceil(b/64) <= (a+b)/64 - a/64 + 1
    } else {
        batch = seq, row = 0, rows = p.rows, slot = seq * p.chunks;
    }
}

// The chunk at a place.
__device__ __forceinline__ DeltaChunk delta_chunk(const DeltaParams &p, int64_t slot) {
    DeltaChunk c;
    int64_t first;
    if (p.offsets) {
        // the last sequence whose first place is not past this one
        int64_t lo = 0, hi = p.sequences;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (min(int64_t(p.offsets[mid]), p.rows) / kChunk + mid <= slot) lo = mid;
            else hi = mid;
        }
        c.seq = lo;
    } else {
        c.seq = slot / p.chunks;
    }
    int64_t rows;
    delta_sequence(p, c.seq, c.batch, c.row, rows, first);
    const int64_t at = (slot - first) * kChunk;
    c.row += at;
    c.rows = at < 0 || at >= rows ? 0 : int(min(rows - at, int64_t(kChunk)));
    return c;
}

template <class T>
__device__ __forceinline__ T *delta_at(const DeltaRows &r, int64_t batch, int64_t row, int head) {
    return reinterpret_cast<T *>(r.data) + batch * r.batch + row * r.row + head * r.head;
}

template <class T>
__device__ __forceinline__ float delta_beta(const DeltaParams &p, int64_t batch, int64_t row, int head) {
    return p.beta_f32 ? *delta_at<float>(p.beta, batch, row, head) : to_f32<T>(*delta_at<T>(p.beta, batch, row, head));
}

__device__ __forceinline__ float delta_g(const DeltaRows &g, int64_t batch, int64_t row, int head) {
    if (!g.data) return 0.0f;
    const float v = *delta_at<float>(g, batch, row, head);
    return v < kLeastDecay ? kLeastDecay : v;  // a NaN stays one
}

// A sum in two f32: differences of sums far from 0 keep their last bits.
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 sum2_add(Sum2 a, Sum2 b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
    const float h = s + e;
    return {h, e - (h - s)};
}
__device__ __forceinline__ float sum2_less(Sum2 a, Sum2 b) { return (a.hi - b.hi) + (a.lo - b.lo); }

// Running sums of a chunk's log decays, by one warp: lane l has rows l and l + 32.
__device__ __forceinline__ void delta_sums(Sum2 (&sum)[2], const float (&g)[2]) {
    const int lane = threadIdx.x % 32;
    sum[0] = {g[0], 0.0f}, sum[1] = {g[1], 0.0f};
#pragma unroll
    for (int o = 1; o < 32; o *= 2)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Sum2 before = {__shfl_up_sync(0xffffffffu, sum[i].hi, o), __shfl_up_sync(0xffffffffu, sum[i].lo, o)};
            if (lane >= o) sum[i] = sum2_add(before, sum[i]);
        }
    const Sum2 half = {__shfl_sync(0xffffffffu, sum[0].hi, 31), __shfl_sync(0xffffffffu, sum[0].lo, 31)};
    sum[1] = sum2_add(half, sum[1]);
}

// 16 bytes to shared memory without a register between; `bytes` of them are
// read, the rest are zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Pieces of bf16 that hold a T: a bf16 itself, or the two that keep 17 bits of
// an f32 and all 11 of an f16.
template <class T>
constexpr int kPieces = 2;
template <>
constexpr int kPieces<__nv_bfloat16> = 1;

// Eight neighbouring elements of a row, zeros past its `left` elements.
template <class T, bool kWide>
__device__ __forceinline__ void load_eight(float (&f)[8], const T *p, int left) {
    if (kWide && left >= 8) {
        load_f32<8>(f, p);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = j < left ? to_f32<T>(p[j]) : 0.0f;
    }
}
__device__ __forceinline__ void store_pieces(char *hi, char *lo, uint32_t at, const float (&f)[8]) {
    uint4 h, l;
    split2(f[0], f[1], h.x, l.x), split2(f[2], f[3], h.y, l.y), split2(f[4], f[5], h.z, l.z), split2(f[6], f[7], h.w, l.w);
    *reinterpret_cast<uint4 *>(hi + at) = h;
    if (lo) *reinterpret_cast<uint4 *>(lo + at) = l;
}

// Rows of a head into tiles of kRows rows and kWidth columns, from row `first`
// of the tile on: 64 rows, zeros past the chunk's `n` and past `dim` columns.
// The second piece lies `lo` bytes behind the first.  By kThreads threads.
// `wide`: the rows are whole 16-byte pieces.
template <class T, int kRows, int kWidth, int kThreads>
__device__ __forceinline__ void load_tile(int thread, char *tile, uint32_t lo, int first, const DeltaRows &r, int64_t batch,
                                          int64_t row, int head, int n, int dim, bool wide) {
    const T *src = delta_at<T>(r, batch, row, head);
#pragma unroll 4
    for (int e = thread; e < kChunk * kWidth / 8; e += kThreads) {
        const int i = e / (kWidth / 8), c = e % (kWidth / 8), left = i < n ? dim - c * 8 : 0;
        const uint32_t at = uint32_t(c / 8 * kRows) * kTileRow + tile_piece(uint32_t(first + i), uint32_t(c % 8));
        const T *from = src + int64_t(left > 0 ? i : 0) * r.row + (left > 0 ? c * 8 : 0);
        if (kPieces<T> == 1 && wide) {
            copy16(smem_addr(tile + at), from, left > 0 ? 16u : 0u);
        } else {
            float f[8];
            if (wide) load_eight<T, true>(f, from, left);
            else load_eight<T, false>(f, from, left);
            store_pieces(tile, kPieces<T> == 2 ? tile + lo : nullptr, at, f);
        }
    }
}

}  // namespace dwp
