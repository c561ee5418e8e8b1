// Checks that the C entry points of the sequence operators share: sizes,
// strides, alignment, overlap and the scratch of the two-call pattern.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "launch.h"

namespace dwp {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;  // batch * rows
constexpr int64_t kMaxChannels = int64_t(1) << 17;
constexpr int64_t kMaxGroups = 1024;
constexpr int64_t kMaxSegments = (int64_t(1) << 30) - 2;
constexpr int64_t kMaxStates = 128;
constexpr int64_t kMaxWidth = 8;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxSpan = int64_t(1) << 58;  // elements from a tensor's first row to its last, each way

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round16(size_t n) { return (n + 15u) / 16u * 16u; }

inline bool dtype_ok(int64_t t) { return t == DWP_F32 || t == DWP_BF16 || t == DWP_F16; }
inline int64_t size_of(int64_t t) { return t == DWP_F32 ? 4 : 2; }
inline bool aligned(const void *p, int64_t n) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(n - 1)) == 0; }

// Bytes that a tensor of rows covers: `rows` pieces of `width` bytes, `row`
// bytes apart, in each of `batch` entries `step` bytes apart.
struct Region {
    uintptr_t at;
    int64_t batch, rows, width, step, row;
    // The same bytes, the smaller stride (or the only one) going by rows: one
    // row a batch entry, and rows that lie outside the batch, are compared too.
    Region by_rows() const {
        if (rows > 1 && (batch == 1 || row <= step)) return *this;
        return {at, rows, batch, width, row, step};
    }
    bool empty() const { return at == 0 || batch <= 0 || rows <= 0 || width <= 0; }
    uintptr_t end() const { return at + uintptr_t((batch - 1) * step + (rows - 1) * row + width); }
    bool regular() const { return batch == 1 || step % row == 0; }
};

inline Region flat(const void *p, int64_t bytes) {
    return {reinterpret_cast<uintptr_t>(p), 1, 1, bytes, bytes, bytes};
}

inline bool overlap(const Region &a, const Region &b) {
    if (a.empty() || b.empty() || a.end() <= b.at || b.end() <= a.at) return false;
    // column ranges of one wider tensor: apart in every row
    if (a.row == b.row && a.row > 0 && a.regular() && b.regular() && (a.rows > 1 || a.batch > 1) &&
        (b.rows > 1 || b.batch > 1)) {
        const uintptr_t lo = a.at < b.at ? a.at : b.at, hi = a.at < b.at ? b.at : a.at;
        const int64_t d = int64_t((hi - lo) % uintptr_t(a.row));
        const int64_t wl = a.at < b.at ? a.width : b.width, wh = a.at < b.at ? b.width : a.width;
        if (d >= wl && d + wh <= a.row) return false;
    }
    return true;
}

// Regions of one call: outputs must overlap nothing else.
struct Regions {
    static constexpr int kMost = 32;
    Region r[kMost];
    bool out[kMost];
    int n = 0;
    void in(const Region &x) { r[n] = x, out[n++] = false; }
    void output(const Region &x) { r[n] = x, out[n++] = true; }
    bool clash() const {
        for (int i = 0; i < n; ++i)
            for (int j = i + 1; j < n; ++j)
                if ((out[i] || out[j]) && overlap(r[i], r[j])) return true;
        return false;
    }
};

// Checks, and the alignment that a call's tensors have in common.
struct Check {
    dwp_status status = DWP_SUCCESS;
    // every address and byte stride seen, or-ed: of the rows, of B and C, of f32 states
    uintptr_t bits = 0, bits_bc = 0, bits_state = 0;
    Regions regions;

    void fail(dwp_status s) {
        if (status == DWP_SUCCESS) status = s;
    }
    void require(bool ok) {
        if (!ok) fail(DWP_ERR_INVALID_VALUE);
    }
    // rows of `inner` elements of type t
    void rows(const dwp_rows &x, int64_t t, int64_t batch, int64_t n, int64_t inner, bool output, bool track = true) {
        const int64_t e = size_of(t);
        require(x.data != nullptr);
        if (status != DWP_SUCCESS) return;
        if (!aligned(x.data, e)) return fail(DWP_ERR_MISALIGNED);
        // one row (or one batch entry) needs no stride
        const int64_t row = n > 1 ? x.row_stride : inner, step = batch > 1 ? x.batch_stride : inner;
        require(row >= inner && row <= kMaxStride && step >= inner && step <= kMaxStride);
        // and what they span is counted in 64 bits below
        if (status == DWP_SUCCESS) require(n - 1 <= kMaxSpan / row && batch - 1 <= kMaxSpan / step);
        if (status != DWP_SUCCESS) return;
        // rows of an output may not fold onto one another
        if (output && batch > 1 && n > 1)
            require(step >= (n - 1) * row + inner || row >= (batch - 1) * step + inner);
        if (status != DWP_SUCCESS) return;
        bits |= reinterpret_cast<uintptr_t>(x.data) | uintptr_t(row * e) | uintptr_t(step * e);
        if (track) {
            const Region r{reinterpret_cast<uintptr_t>(x.data), batch, n, inner * e, step * e, row * e};
            output ? regions.output(r.by_rows()) : regions.in(r.by_rows());
        }
    }
    // rows of `count` heads of `inner` elements: checked as rows of their whole
    // span, what lies between the heads counted in
    void heads(const dwp_heads &x, int64_t t, int64_t batch, int64_t n, int64_t count, int64_t inner, bool output) {
        require(count == 1 || (x.head_stride >= inner && x.head_stride <= kMaxStride));
        if (status != DWP_SUCCESS) return;
        const dwp_rows r{x.data, x.batch_stride, x.row_stride};
        rows(r, t, batch, n, (count > 1 ? (count - 1) * x.head_stride : 0) + inner, output);
        if (count > 1) bits |= uintptr_t(x.head_stride * size_of(t));
    }
    // dense array of `count` elements of type t; NULL allowed if optional
    void dense(const void *p, int64_t t, int64_t count, bool output, bool optional, uintptr_t *seen = nullptr) {
        if (!optional && count > 0) require(p != nullptr);
        if (status != DWP_SUCCESS || !p) return;
        if (!aligned(p, size_of(t))) return fail(DWP_ERR_MISALIGNED);
        if (seen) *seen |= reinterpret_cast<uintptr_t>(p);
        const Region r = flat(p, count * size_of(t));
        output ? regions.output(r) : regions.in(r);
    }
    // Rows of `inner` elements of type t are whole 16-byte pieces.
    bool wide(int64_t inner, int64_t t) const { return ((bits | uintptr_t(inner * size_of(t))) & 15u) == 0; }
    // The scratch of the two-call pattern; true: go on and launch.  A call that
    // needs none asks for 16 bytes: of 0 a caller's allocation may be NULL, and
    // the second call would be taken for another query.
    bool scratch(void *p, size_t *bytes, size_t need, dwp_status *st) {
        if (need < 16u) need = 16u;
        if (status != DWP_SUCCESS) return *st = status, false;
        if (!p) return *bytes = need, *st = DWP_SUCCESS, false;
        if (*bytes < need) return *st = DWP_ERR_SCRATCH_TOO_SMALL, false;
        if (!aligned(p, 16)) return *st = DWP_ERR_MISALIGNED, false;
        regions.output(flat(p, int64_t(need)));
        if (regions.clash()) return *st = DWP_ERR_ALIASING, false;
        return true;
    }
};

inline dwp_status launched(cudaError_t err) {
    if (err == cudaSuccess) return DWP_SUCCESS;
    cudaGetLastError();
    return DWP_ERR_CUDA;
}

// Sizes common to calls over packed or batched rows; the number of sequences.
inline int64_t sequences(Check &c, int64_t channels, int64_t batch, int64_t rows, int64_t segments, const void *offsets) {
    c.require(channels >= 1 && channels <= kMaxChannels && batch >= 0 && rows >= 0 && batch <= kMaxRows &&
              rows <= kMaxRows);
    if (c.status != DWP_SUCCESS) return 0;
    c.require(batch * rows <= kMaxRows);
    if (offsets) {
        c.require(batch == 1 && segments >= 0 && segments <= kMaxSegments);
        if (!aligned(offsets, 4)) c.fail(DWP_ERR_MISALIGNED);
        if (c.status == DWP_SUCCESS) c.regions.in(flat(offsets, (segments + 1) * 4));
        return segments;
    }
    c.require(segments == 0);
    return batch;
}

// A state cache's slots.
inline void check_slots(Check &c, const void *state, int64_t t, int64_t batch, int64_t num_slots, int64_t stride,
                 int64_t inner, const int32_t *slots) {
    c.require(num_slots >= 0 && num_slots <= kMaxRows && (slots || num_slots >= batch));
    if (slots && !aligned(slots, 4)) c.fail(DWP_ERR_MISALIGNED);
    if (c.status == DWP_SUCCESS && slots) c.regions.in(flat(slots, batch * 4));
    if (inner > 0 && num_slots > 0) {
        dwp_rows r{const_cast<void *>(state), 0, stride};
        c.rows(r, t, 1, num_slots, inner, true);
    }
}

}  // namespace dwp
