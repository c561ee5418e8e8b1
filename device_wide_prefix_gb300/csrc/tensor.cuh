// Matrix products on the fifth-generation tensor cores: shared-memory tiles,
// their descriptors, tensor memory and its accesses.
//
// A tile is rows of 64 bf16 (128 bytes), its 16-byte pieces exchanged within
// each eight rows (piece c of row r lies at c ^ (r % 8)), at an address that
// is a multiple of 1024.  A wider matrix is several tiles side by side.  The
// same tile serves a product whose inner index runs along the rows ("inner")
// or from row to row ("outer"), by its descriptor alone.
//
// Every product has 128 rows of D, one for each lane of tensor memory; a
// warp reads and writes the 32 lanes of its place in its group of four.
#pragma once

#include "device.cuh"

namespace dwp {

constexpr uint32_t kTileRow = 128;  // bytes

// Offset of 16-byte piece `c` of row `r` in a tile.
__device__ __forceinline__ uint32_t tile_piece(uint32_t r, uint32_t c) { return r * kTileRow + ((c ^ (r & 7u)) << 4); }
// Offset of element `j` of row `r`, in a matrix of tiles of `rows` rows.
__device__ __forceinline__ uint32_t tile_at(uint32_t r, uint32_t j, uint32_t rows) {
    return j / 64u * rows * kTileRow + tile_piece(r, j % 64u / 8u) + j % 8u * 2u;
}

// Shared-memory descriptor: 128-byte exchange, eight-row groups 1024 bytes
// apart; `step`: bytes between blocks of 64 along an outer operand's rows.
__device__ __forceinline__ uint64_t tile_descriptor(uint32_t addr, uint32_t step) {
    return uint64_t((addr & 0x3ffffu) >> 4) | uint64_t(step >> 4) << 16 | uint64_t(1024u >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor: bf16 operands, f32 sums, 128 x n; whether A and B
// are outer.
__device__ __forceinline__ uint32_t product_kind(int n, bool a_outer, bool b_outer) {
    return 1u << 4 | 1u << 7 | 1u << 10 | uint32_t(a_outer) << 15 | uint32_t(b_outer) << 16 | uint32_t(n / 8) << 17 | 8u << 24;
}

// D (+)= A B, 16 of the inner index.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"(uint32_t(add))
        : "memory");
}
// The same with A in tensor memory: two values of the inner index a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(kind), "r"(uint32_t(add))
        : "memory");
}

// An operand in shared memory, in tiles of kRows rows.
template <int kRows, bool kOuter>
struct Operand {
    uint64_t first;
    __device__ __forceinline__ explicit Operand(const void *tiles)
        : first(tile_descriptor(smem_addr(tiles), kOuter ? kRows * kTileRow : 16u)) {}
    // of sixteen inner indices: the address is the descriptor's low part
    __device__ __forceinline__ uint64_t at(int k) const {
        return first + (kOuter ? k * 16 * kTileRow : k / 4 * kRows * kTileRow + k % 4 * 32) / 16;
    }
};

// D (+)= A B over K of the inner index.  By one thread; the loops unroll, so
// that a product is a run of instructions whose descriptors differ by constants.
template <int N, int K, int AR, bool AO, int BR, bool BO>
__device__ __forceinline__ void product_ss(uint32_t d, const Operand<AR, AO> &a, const Operand<BR, BO> &b, bool add) {
    const uint32_t kind = product_kind(N, AO, BO);
#pragma unroll
    for (int i = 0; i < K / 16; ++i) mma_ss(d, a.at(i), b.at(i), kind, add || i > 0);
}
template <int N, int K, int BR, bool BO>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, const Operand<BR, BO> &b, bool add) {
    const uint32_t kind = product_kind(N, false, BO);
#pragma unroll
    for (int i = 0; i < K / 16; ++i) mma_ts(d, a + uint32_t(i) * 8u, b.at(i), kind, add || i > 0);
}

// One thread of a whole warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A warpgroup's registers a thread, from the block's own share: all shares
// together are at most the threads' at launch.
template <int N>
__device__ __forceinline__ void set_registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void set_registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Wait for the phase of the given parity, without sleeping between polls (a
// product takes less than a sleep); false after a second or so (a poll that finds
// nothing takes 3.7 us).
//
// A block whose wait runs out gives up: whoever loads or issues and waited in vain
// arrives nowhere and issues nothing from then on, so that who needs it waits in
// vain too; what the block could not compute is NaN; and the copies and products
// that are still on their way are waited for before it ends.
#ifdef DWP_DELTA_TEST
constexpr uint32_t kProductWaitLimit = 1u << 13;
#else
constexpr uint32_t kProductWaitLimit = 1u << 18;
#endif
__device__ __forceinline__ bool mma_wait(uint64_t *bar, uint32_t parity) {
    for (uint32_t i = 0; i < kProductWaitLimit; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}
__device__ __forceinline__ float not_a_number() { return __int_as_float(0x7fffffff); }

// Places of a kernel that wait, for the build with test hooks.
enum WaitSite {
    kNoSite, kLocalRows, kLocalProduct,
    kIssueRows, kIssueState, kIssueSides, kIssueCorrections, kLoadRoom, kLoadLanded, kDecayRoom,
    kChainRows, kChainKeys, kChainOther, kChainInverse, kChainState, kChainOutputs, kChainRoom, kChainSide,
    kGradFirst, kGradStates, kGradSecond, kGradRows, kGradEnds
};
#ifdef DWP_DELTA_TEST
// A wait at the stalled site, but for the first `skip` of a thread, is for a barrier
// at which nothing arrives.
struct Stall {
    uint64_t *never;
    int site, skip;
    __device__ __forceinline__ bool at(int here) { return here == site && skip-- <= 0 && !mma_wait(never, 0); }
};
#endif

// A box of a tensor to shared memory, completing its bytes on `bar`; from
// column `x`, whose byte offset is a multiple of 16, of head, row and batch.
__device__ __forceinline__ void map_load(void *to, const void *map, uint64_t *bar, int x, int head, int row, int batch) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
            smem_addr(to)),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(head), "r"(row), "r"(batch)
        : "memory");
}

// The products issued so far by this thread arrive on `bar` when done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Tensor memory, by one whole warp.  Only after pdl_wait: a block that holds
// some while it waits for an earlier kernel could keep that kernel's blocks
// from theirs.
__device__ __forceinline__ void tmem_alloc(uint32_t *where, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}

#define DWP_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define DWP_W8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])

// Sixteen columns from `at` on of the warp's lanes, one lane a thread.  tmem_ready() before use.
__device__ __forceinline__ void tmem_load(uint32_t (&v)[16], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15}, [%16];"
                 : DWP_R8(v, 0), DWP_R8(v, 8)
                 : "r"(at));
}
__device__ __forceinline__ void tmem_ready() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Eight columns.
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::DWP_W8(v, 0), "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A pair of f32 in two pieces of bf16 each: hi rounded, lo the rounded rest.
// Together they hold 17 bits, lo's sign among them: |x - hi - lo| <= 2^-17 |x|.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
    const float xh = __uint_as_float(hi << 16), yh = __uint_as_float(hi & 0xffff0000u);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(y - yh), "f"(x - xh));
}

}  // namespace dwp
