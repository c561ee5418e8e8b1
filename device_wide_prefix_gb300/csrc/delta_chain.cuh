// Gated delta rule, the states from chunk to chunk (and the outputs), and the
// walk back for the states' gradients.  A block has one sequence and head.
//
// Forward, a chunk:                          Back, from the last chunk:
//   P  = K S                                   X  = K dS,  Y = A^T dO
//   R  = beta (V - e^G P)                      dU = e^{G_C - G} X + scale Y
//   U  = T R                                   dR = T^T dU
//   S  = e^{G_C} S + K^T e^{G_C - G} U         dS = e^{G_C} dS + scale Q^T e^G dO - K^T beta e^G dR
//   O  = scale (e^G Q S + A U)
//
// All products are taken transposed, so that their 128 rows are the values
// and never a chunk's 64 rows: the state, f32 in registers (a thread has one
// value's row and a quarter of the keys), goes to tensor memory as the first operand
// of the next products, as R and U do, and K, Q, T, A and dO are operands in
// shared memory as they are stored.  What is not itself bf16 is two bf16
// (split2): 17 bits, 2^-17 of a number at most is lost; of two such all four
// products are taken (without the smallest a call took 1% less, and
// the gradient of g was up to a fifth further off).
//
// Sixteen warps do this (with eight, twice the registers and rows each, a chunk
// took 1.2 times as long); of four more one issues the products (a warp that issues
// is held back as long as the products before it run), one loads, and one has
// the decays: they work ahead.  Outputs, and what is kept for the gradient, go
// through shared memory, and the sixteen copy them on while they wait for
// products: one of the four warps is slower at that (instructions that come in
// between the chain's are fetched anew each time; 9,000 cycles a chunk), bulk
// copies are slower still (256 bytes in 83 cycles, 64 KB in 5,000).
//
// What bounds it is that each product needs the one before it: a chunk of 128 x
// 128 forward takes about 5,500 cycles (32768 rows x 32 heads, a block an SM at
// most; 6,900 with 128 blocks), of which the products that wait for one another
// are 1,500; carrying numbers between tensor memory, registers and pieces is the
// rest.  4 x 2048 rows x 32 heads take 117 us; x 16 heads, with what the gradient
// needs kept, 188, and back 170.  Keys up to 64 take half the state (KD 64): 170
// us a call of 4 x 2048 x 32 in place of 191.  bf16 rows of whole 16-byte pieces
// come by tensor maps, a chunk ahead (191); others are read and split by the
// sixteen warps between chunks (off 16 bytes 468, f16 414, f32 438).
//
// Few sequences and heads leave most of the GPU idle while each walks its
// chunks.  A state goes through a part of a sequence linearly, S -> M S + E, so
// such sequences are cut in parts: pass 1 walks the first part and finds E (from
// zeros) and M (from the unit matrix, without values) of those between at the
// same time; their states are joined (delta_join_kernel); pass 2 walks the
// others.  That is two parts' time for the whole sequence's.
#pragma once

#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kChainThreads = 512, kHelpThreads = 128, kIssueWarp = kChainThreads / 32;
constexpr int kParts = kChainThreads / 128, kT = kChunk / kParts;  // kT: a thread's rows of the chunk
// 96 registers a thread at launch, of which the helpers give some to the chain:
// 512 x 104 + 128 x 64 = 640 x 96.
constexpr int kChainRegisters = 104, kHelpRegisters = 64;
constexpr int kMostValues = 128;

// Shared memory: the chunks' inputs, the outputs on their way, and what is kept.
template <class T, int KD, bool kBack, bool kMaps>
struct ChainSpace {
    static constexpr int kP = kPieces<T>;
    static constexpr uint32_t kTileBytes = kChunk * kTileRow;  // of 64 x 64
    static constexpr uint32_t kKeys = kChunk * KD * 2, kValues = kChunk * kMostValues * 2;
    static constexpr uint32_t k = 0, q = k + kP * kKeys, v = q + kP * kKeys;
    static constexpr uint32_t inverse = v + (kBack ? kP * kValues : kChunk * kMostValues * uint32_t(sizeof(T)));
    static constexpr uint32_t weights = inverse + 2 * kTileBytes, bytes = weights + 2 * kTileBytes;
    static constexpr int kStages = kMaps ? 2 : 1;
    // With two stages there is no room for outputs on their way beside the two
    // pieces of the weights and what is kept: they wait where a state would be
    // kept, or, if one is, in the place of a chunk's V, which nothing reads by then.
    static constexpr bool kOutInV = kMaps && !kBack;
    static constexpr uint32_t out = kStages * bytes, kOut = kBack || kOutInV ? 0 : kChunk * kMostValues * uint32_t(sizeof(T));
    static constexpr uint32_t keep = out + kOut, kKeep = 2 * kMostValues * KD * 2;
    static_assert(kKeep >= 2 * kValues, "the corrections fit the kept state's place");
    static constexpr size_t kAll = 1024 + keep + kKeep;
};

// Decays and betas of a chunk's rows.
struct ChainRows {
    alignas(16) float beta[kChunk], first[kChunk], rest[kChunk];  // first: e^G, rest: e^{G_C - G}
};

// A block's part of the walk along its sequence, and what it finds: the whole
// (pass 0, or a part's own outputs), E or M.
template <bool kBack, int kPass>
struct ChainWalk {
    int64_t batch, slot0, part;
    int row0, rows, chunks, last;  // chunks from slot0 on, and the one that a walk back begins at (rows are under 2^31)
    bool unit, whole_part;         // finds M; has outputs of its own
    int values;
    __device__ __forceinline__ explicit ChainWalk(const DeltaParams &p) {
        int64_t row, all;
        delta_sequence(p, blockIdx.x, batch, row, all, slot0);
        part = kPass == 0 ? 0 : kPass == 1 ? (blockIdx.z + 1) / 2 : blockIdx.z + 1;
        unit = kPass == 1 && part > 0 && blockIdx.z % 2 == 0, whole_part = kPass != 1 || part == 0;
        const int64_t all_chunks = (all + kChunk - 1) / kChunk, before = kPass != 0 ? min(part * p.part_chunks, all_chunks) : 0;
        last = int(all_chunks - 1 - before);
        chunks = int(kPass != 0 ? min(p.part_chunks, all_chunks - before) : all_chunks);
        const int64_t skip = kBack ? 0 : before;
        row0 = int(row + skip * kChunk), rows = int(all - skip * kChunk), slot0 += skip;
        values = unit ? p.keys : p.values;
    }
    __device__ __forceinline__ int chunk_of(int step) const { return kBack ? last - step : step; }
    __device__ __forceinline__ int rows_in(int c) const { return min(rows - c * kChunk, kChunk); }
    // Where the state at its end goes: the last part's is the sequence's, another's own is the next one's start.
    __device__ __forceinline__ float *end_state(const DeltaBackwardParams &bp) const {
        const DeltaParams &p = bp.f;
        const bool last = kPass == 0 || (kPass == 2 && part + 1 == p.parts);
        float *to = last ? kBack ? bp.grad_initial : p.final : unit ? p.part_maps : kPass == 1 ? p.part_ends : nullptr;
        int64_t place = last ? int64_t(blockIdx.x) * p.heads + blockIdx.y : (blockIdx.x * p.parts + part) * p.heads + blockIdx.y;
        if (kPass == 1 && part == 0) to = p.part_starts, place += p.heads;
        return to ? to + place * p.keys * values : nullptr;
    }
};

// Of a walk in which a wait was in vain: NaN in all that it writes.  By the whole block.
template <class T, int KD, bool kBack, int kPass>
__device__ __noinline__ void chain_give_up(const DeltaBackwardParams &bp) {
    constexpr int kThreads = kChainThreads + kHelpThreads;
    const DeltaParams &p = bp.f;
    const ChainWalk<kBack, kPass> walk(p);
    const int tid = threadIdx.x, head = blockIdx.y, values = walk.values, tiles = (values + 63) / 64;
    auto fill = [&](float *to, int words) {
        for (int e = tid; e < words; e += kThreads) to[e] = __uint_as_float(0xffffffffu);  // in pairs of bf16 too
    };
    float *kept = kBack ? bp.ends : p.states, *kept_rows = kBack ? bp.dr : p.u;
    for (int step = 0; walk.whole_part && kept && step < walk.chunks; ++step) {
        const int64_t at = (walk.slot0 + walk.chunk_of(step)) * p.heads + head;
        fill(kept + at * KD * values, KD * values);
        fill(kept_rows + at * kChunk * 64 * tiles, kChunk * 64 * tiles);
    }
    for (int step = 0; !kBack && walk.whole_part && step < walk.chunks; ++step) {
        const int c = walk.chunk_of(step);
        T *to = delta_at<T>(p.out, walk.batch, walk.row0 + c * kChunk, head);
        for (int e = tid; e < walk.rows_in(c) * values; e += kThreads)
            to[e / values * p.out.row + e % values] = from_f32<T>(not_a_number());
    }
    if (float *to = walk.end_state(bp)) fill(to, p.keys * values);
}

// kMaps: bf16 rows of whole 16-byte pieces, which come by tensor maps.  kPass: 0,
// or 1 and 2 over parts of sequences (what a block finds in pass 1, asked in
// every chunk, makes a chunk 1.25 times as long).
template <class T, int KD, bool kBack, bool kMaps, int kPass>
__global__ void __launch_bounds__(kChainThreads + kHelpThreads, 1)
    delta_chain_kernel(const __grid_constant__ DeltaBackwardParams bp, const __grid_constant__ DeltaMaps maps) {
    using Space = ChainSpace<T, KD, kBack, kMaps>;
    constexpr int kP = Space::kP, kH = KD / kParts, kStages = Space::kStages;  // kH: keys of a thread
    extern __shared__ char raw[];
    __shared__ ChainRows rows_of[2];
    __shared__ uint64_t done[5], ready[3], full[2], empty[2], landed[2], drained;
    __shared__ uint32_t tmem, in_vain;
    const DeltaParams &p = bp.f;
    char *sm = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
    const int head = blockIdx.y, kh = head / (p.heads / p.key_heads), keys = p.keys;
    const int64_t seq = blockIdx.x;
    const ChainWalk<kBack, kPass> walk(p);
    constexpr bool kCut = kPass != 0;
    const int64_t batch = walk.batch, slot0 = walk.slot0, part = walk.part;
    const int row0 = walk.row0, chunks = walk.chunks;
    const bool unit = walk.unit, whole_part = walk.whole_part;
    const int values = walk.values;
    auto chunk_of = [&](int step) { return walk.chunk_of(step); };
    auto rows_in = [&](int c) { return walk.rows_in(c); };
    auto stage_of = [&](int step) { return kStages == 2 ? step & 1 : 0; };
    auto round_of = [&](int step) { return uint32_t(step) / kStages & 1u; };
    float *const kept = whole_part ? kBack ? bp.ends : p.states : nullptr, *const kept_rows = kBack ? bp.dr : p.u;

#ifdef DWP_DELTA_TEST
    __shared__ uint64_t never;
    if (tid == 0) mbar_init(&never, 1);
    Stall stall{&never, p.stall_site, p.stall_skip};
#endif
    if (tid == 0) {
        in_vain = 0;
        for (int i = 0; i < 5; ++i) mbar_init(&done[i], 1);
        // one arrival a warp: 256 on one word take a thousand cycles
        for (int i = 0; i < 3; ++i) mbar_init(&ready[i], kChainThreads / 32);
        // the planes and boxes, the decays, and, without maps, the chain's own loads
        for (int i = 0; i < 2; ++i)
            mbar_init(&landed[i], 1), mbar_init(&full[i], kMaps ? 2 : 2 + kChainThreads / 32),
                mbar_init(&empty[i], Space::kOutInV ? 1 + kChainThreads / 32 : 1);  // the products; and outputs that waited there
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem, 512);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // columns: sums of the first product; of the second; of the state's; then
    // operands: the state (hi, lo), R or U (hi, lo), U as it is or the queries' side (hi, lo)
    const uint32_t tm = tmem;
    constexpr uint32_t kD0 = 0, kD1 = 64, kDS = 128, kS = 256, kR = 384, kU = 448;
    // No wait of this thread was in vain.  Where one was, a helper arrives nowhere and
    // issues nothing more; the chain's threads go on to the walk's end, where they
    // ask one another (asked each chunk, a walk took 1 to 6% longer).
    bool ok = true;
    auto wait = [&](uint64_t &bar, uint32_t parity, [[maybe_unused]] WaitSite site) {
#ifdef DWP_DELTA_TEST
        if (ok && stall.at(site)) ok = false;
#endif
        if (ok) ok = mma_wait(&bar, parity & 1u);
    };

    if (warp >= kIssueWarp) set_registers_down<kHelpRegisters>();
    else set_registers_up<kChainRegisters>();
    if (warp == kIssueWarp) {
        const bool one = elect_one();
        for (int step = 0; step < chunks; ++step) {
            const int st = stage_of(step);
            char *s = sm + st * Space::bytes;
            const Operand<kChunk, true> Ko(s + Space::k), Klo(s + Space::k + Space::kKeys);
            wait(full[st], round_of(step), kIssueRows);
            wait(ready[0], uint32_t(step), kIssueState);
            tmem_fence_after();
            if (one && ok) {
                const Operand<kChunk, false> K(s + Space::k), Kl(s + Space::k + Space::kKeys);
                product_ts<kChunk, KD>(tm + kD0, tm + kS, K, false);
                product_ts<kChunk, KD>(tm + kD0, tm + kS + KD / 2, K, true);
                if constexpr (kP == 2) {
                    product_ts<kChunk, KD>(tm + kD0, tm + kS, Kl, true);
                    product_ts<kChunk, KD>(tm + kD0, tm + kS + KD / 2, Kl, true);
                }
                mma_commit(&done[0]);
                if constexpr (kBack) {
                    const Operand<kChunk, true> dO(s + Space::v), dOl(s + Space::v + Space::kValues), A(s + Space::weights),
                        Al(s + Space::weights + Space::kTileBytes);
                    if (!unit) product_ss<kChunk, kChunk>(tm + kD1, dO, A, false);
                    if (!unit) product_ss<kChunk, kChunk>(tm + kD1, dO, Al, true);
                    if constexpr (kP == 2) {
                        if (!unit) {
                            product_ss<kChunk, kChunk>(tm + kD1, dOl, A, true);
                            product_ss<kChunk, kChunk>(tm + kD1, dOl, Al, true);
                        }
                    }
                } else if (whole_part) {
                    const Operand<kChunk, false> Q(s + Space::q), Ql(s + Space::q + Space::kKeys);
                    product_ts<kChunk, KD>(tm + kDS, tm + kS, Q, false);
                    product_ts<kChunk, KD>(tm + kDS, tm + kS + KD / 2, Q, true);
                    if constexpr (kP == 2) {
                        product_ts<kChunk, KD>(tm + kDS, tm + kS, Ql, true);
                        product_ts<kChunk, KD>(tm + kDS, tm + kS + KD / 2, Ql, true);
                    }
                }
                mma_commit(&done[1]);
            }
            __syncwarp();
            wait(ready[1], uint32_t(step), kIssueSides);
            tmem_fence_after();
            if (one && ok) {
                const Operand<kChunk, kBack> inv(s + Space::inverse), invl(s + Space::inverse + Space::kTileBytes);
                product_ts<kChunk, kChunk>(tm + kD0, tm + kR, inv, false);
                product_ts<kChunk, kChunk>(tm + kD0, tm + kR + 32, inv, true);
                product_ts<kChunk, kChunk>(tm + kD0, tm + kR, invl, true);
                product_ts<kChunk, kChunk>(tm + kD0, tm + kR + 32, invl, true);
                mma_commit(&done[2]);
            }
            __syncwarp();
            wait(ready[2], uint32_t(step), kIssueCorrections);
            tmem_fence_after();
            if (one && ok) {
                product_ts<KD, kChunk>(tm + kDS, tm + kR, Ko, false);
                product_ts<KD, kChunk>(tm + kDS, tm + kR + 32, Ko, true);
                if constexpr (kP == 2) {
                    product_ts<KD, kChunk>(tm + kDS, tm + kR, Klo, true);
                    product_ts<KD, kChunk>(tm + kDS, tm + kR + 32, Klo, true);
                }
                if (kBack && !unit) {
                    const Operand<kChunk, true> Q(s + Space::q), Ql(s + Space::q + Space::kKeys);
                    product_ts<KD, kChunk>(tm + kDS, tm + kU, Q, true);
                    product_ts<KD, kChunk>(tm + kDS, tm + kU + 32, Q, true);
                    if constexpr (kP == 2) {
                        product_ts<KD, kChunk>(tm + kDS, tm + kU, Ql, true);
                        product_ts<KD, kChunk>(tm + kDS, tm + kU + 32, Ql, true);
                    }
                }
                mma_commit(&done[3]);
                if (!kBack && whole_part) {
                    const Operand<kChunk, false> A(s + Space::weights), Al(s + Space::weights + Space::kTileBytes);
                    product_ts<kChunk, kChunk>(tm + kD1, tm + kU, A, false);
                    product_ts<kChunk, kChunk>(tm + kD1, tm + kU + 32, A, true);
                    product_ts<kChunk, kChunk>(tm + kD1, tm + kU, Al, true);
                    // (the smallest product is at most 2^-16 of a term: nothing to a bf16 output)
                    if constexpr (kP == 2) product_ts<kChunk, kChunk>(tm + kD1, tm + kU + 32, Al, true);
                    mma_commit(&done[4]);
                }
                mma_commit(&empty[st]);
            }
            __syncwarp();
        }
        // however the walk ended, no product is on its way after this
        if (one) mma_commit(&drained);
        mma_wait(&drained, 0);
        __syncwarp();
    } else if (warp > kIssueWarp) {
        const bool loads = warp == kIssueWarp + 1, decays = warp == kIssueWarp + 2;
        // A chunk's copies, and, when they have landed, word of it.  `asked`: they were issued.
        auto load = [&](int step) {
            const int st = stage_of(step);
            const int c = chunk_of(step), row = row0 + c * kChunk;
            const int64_t at = (slot0 + c) * p.heads + head;
            char *s = sm + st * Space::bytes;
            if (step >= kStages) wait(empty[st], round_of(step) + 1u, kLoadRoom);
            constexpr uint32_t planes = 4 * Space::kTileBytes;
            constexpr uint32_t boxes = kMaps ? 2 * Space::kKeys + Space::kValues : 0;
            const bool asked = __shfl_sync(0xffffffffu, ok, 0);
            if (lane == 0 && asked) {
                uint64_t *bar = &landed[st];
                mbar_arrive_expect_tx(bar, planes + boxes);
                bulk_load(s + Space::inverse, p.inverse + at * kChunk * kChunk, 2 * Space::kTileBytes, bar);
                bulk_load(s + Space::weights, p.weights + at * kChunk * kChunk, 2 * Space::kTileBytes, bar);
                if constexpr (kMaps) {
                    const int r = row, b = int(batch);
#pragma unroll
                    for (int x = 0; x < KD; x += 64) {
                        map_load(s + Space::k + x * kTileRow, &maps.k, bar, x, kh, r, b);
                        map_load(s + Space::q + x * kTileRow, &maps.q, bar, x, kh, r, b);
                    }
                    if constexpr (kBack) {
                        map_load(s + Space::v, &maps.v, bar, 0, head, r, b);
                        map_load(s + Space::v + 64 * kTileRow, &maps.v, bar, 64, head, r, b);
                    } else {
                        map_load(s + Space::v, &maps.v, bar, 0, head, r, b);
                    }
                }
            }
            return asked;
        };
        auto landing = [&](int step, bool asked) {
            const int st = stage_of(step), n = rows_in(chunk_of(step));
            // what was asked for is waited for, whatever else was in vain
            bool here = asked && mma_wait(&landed[st], round_of(step));
#ifdef DWP_DELTA_TEST
            if (stall.at(kLoadLanded)) here = false;
#endif
            if (!__all_sync(0xffffffffu, here)) {
                ok = false;
                return;
            }
            if constexpr (kMaps) {
                // the rows after a short chunk's are another sequence's: they are made zeros before they count
                if (n < kChunk) {
                    char *s = sm + st * Space::bytes;
                    // rows of 128 bytes in tiles; of 256 in the values' forward
                    auto clear = [&](char *tile, uint32_t pitch) {
                        for (uint32_t e = uint32_t(n) * pitch / 16 + lane; e < kChunk * pitch / 16; e += 32)
                            reinterpret_cast<uint4 *>(tile)[e] = make_uint4(0, 0, 0, 0);
                    };
                    for (int x = 0; x < KD; x += 64) clear(s + Space::k + x * kTileRow, 128), clear(s + Space::q + x * kTileRow, 128);
                    if constexpr (kBack) clear(s + Space::v, 128), clear(s + Space::v + 64 * kTileRow, 128);
                    else clear(s + Space::v, 256);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
        };
        float g[2], b[2];
        auto read_decays = [&](int step) {
            const int c = chunk_of(step), row = row0 + c * kChunk;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane + 32 * i;
                g[i] = r < rows_in(c) ? delta_g(p.g, batch, row + r, head) : 0.0f;
                b[i] = r < rows_in(c) ? delta_beta<T>(p, batch, row + r, head) : 0.0f;
            }
        };
        auto put_decays = [&](int step) {
            const int st = stage_of(step);
            if (step >= kStages) wait(empty[st], round_of(step) + 1u, kDecayRoom);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                return;
            }
            ChainRows &r = rows_of[st];
            Sum2 sum[2];
            delta_sums(sum, g);
            const Sum2 last = {__shfl_sync(0xffffffffu, sum[1].hi, 31), __shfl_sync(0xffffffffu, sum[1].lo, 31)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float e = __expf(sum[i].hi);
                r.beta[lane + 32 * i] = b[i], r.first[lane + 32 * i] = fmaf(e, sum[i].lo, e);
                r.rest[lane + 32 * i] = __expf(sum2_less(last, sum[i]));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
        };
        // the first stages at once, then each as it is free
        const int first = min(chunks, kStages);
        if (loads) {
            bool asked[2] = {};
            for (int step = 0; step < first; ++step) asked[step] = load(step);
            for (int step = 0; step < first; ++step) landing(step, asked[step]);
            for (int step = first; step < chunks; ++step) landing(step, load(step));
        }
        if (decays)
            for (int step = 0; step < chunks; ++step) read_decays(step), put_decays(step);
    } else {
        const int quarter = warp / 4, dv = warp % 4 * 32 + lane, t0 = quarter * kT, k0 = quarter * kH;
        const uint32_t mine = tm + (uint32_t(warp % 4) << 21);
        float S[kH];
        {
            const float *from = !kCut || part == 0 ? kBack ? bp.grad_final : p.initial : whole_part ? p.part_starts : nullptr;
            const int64_t at = (!kCut || part == 0 ? seq * p.heads + head : (seq * p.parts + part) * p.heads + head) * keys * values + dv;
#pragma unroll
            for (int k = 0; k < kH; ++k) {
                S[k] = from && dv < values && k0 + k < keys ? from[at + int64_t(k0 + k) * values] : 0.0f;
                if (unit && k0 + k == dv && dv < keys) S[k] = 1.0f;
            }
        }
        // what was stored is there for the products, and the copies
        auto arrive = [&](int which) {
            tmem_stored();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[which]);
        };
        auto wait_done = [&](int which, int step) {
            wait(done[which], uint32_t(step), WaitSite(kChainKeys + which));
            tmem_fence_after();
        };
        auto read = [&](float (&x)[kT], uint32_t at) {
            uint32_t v[kT];
            tmem_load(v, mine + at);
            tmem_ready();
#pragma unroll
            for (int j = 0; j < kT; ++j) x[j] = __uint_as_float(v[j]);
        };
        // numbers of this thread's rows of the chunk, in two pieces, as an operand
        auto put_rows = [&](uint32_t at, const float (&x)[kT]) {
            uint32_t hi[kT / 2], lo[kT / 2];
#pragma unroll
            for (int j = 0; j < kT / 2; ++j) split2(x[2 * j], x[2 * j + 1], hi[j], lo[j]);
            tmem_store(mine + at + quarter * (kT / 2), hi);
            tmem_store(mine + at + 32 + quarter * (kT / 2), lo);
        };
        auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(kChainThreads) : "memory"); };
        // the same, and whether no wait of any of the threads was in vain
        auto all_well = [&] {
            uint32_t all;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(all)
                         : "r"(uint32_t(ok)), "n"(kChainThreads)
                         : "memory");
            return all != 0;
        };
        // from shared to global memory, whole 16-byte pieces
        auto copy = [&](char *to, const char *from, int bytes) {
#pragma unroll 4
            for (int e = tid * 16; e < bytes; e += kChainThreads * 16)
                *reinterpret_cast<uint4 *>(to + e) = *reinterpret_cast<const uint4 *>(from + e);
        };
        auto copy_state = [&](int64_t at) {
            for (int i = 0; i < 2 * KD / 64; ++i)
                copy(reinterpret_cast<char *>(kept + at * KD * values) + int64_t(i) * values * kTileRow,
                     sm + Space::keep + i * kMostValues * kTileRow, values * int(kTileRow));
        };
        auto copy_rows = [&](int64_t at) {
            const int tiles = (values + 63) / 64;
            for (int i = 0; i < 2; ++i)
                copy(reinterpret_cast<char *>(kept_rows + at * kChunk * 64 * tiles) + i * tiles * int(Space::kTileBytes),
                     sm + Space::keep + i * Space::kValues, tiles * int(Space::kTileBytes));
        };
        // where the outputs of chunk `step` wait while the next chunk is taken
        auto out_place = [&](int step) {
            return reinterpret_cast<T *>(sm + (Space::kOutInV && kept ? stage_of(step + 1) * Space::bytes + Space::v : Space::out));
        };
        auto copy_out = [&](int step) {
            const int c = chunk_of(step);
            const int n = rows_in(c);
            const T *from = out_place(step);
            T *to = delta_at<T>(p.out, batch, row0 + c * kChunk, head);
            if (p.out_wide) {
                constexpr int kEach = 16 / int(sizeof(T)), kRow = kMostValues / kEach;
                const int j = tid % kRow * kEach;
                if (j < values)
#pragma unroll 4
                    for (int i = tid / kRow; i < n; i += kChainThreads / kRow)
                        *reinterpret_cast<uint4 *>(to + i * p.out.row + j) =
                            *reinterpret_cast<const uint4 *>(from + i * kMostValues + j);
            } else {
                const int j = tid % kMostValues;
                if (j < values)
                    for (int i = tid / kMostValues; i < n; i += kChainThreads / kMostValues)
                        to[i * p.out.row + j] = from[i * kMostValues + j];
            }
        };
        // Rows that no map brings (in two pieces of bf16, or off 16 bytes): by all
        // threads, between chunks, into the one stage.
        auto load_rows = [&](int step) {
            const int c = chunk_of(step), row = row0 + c * kChunk;
            const int n = rows_in(c);
            load_tile<T, kChunk, KD, kChainThreads>(tid, sm + Space::k, Space::kKeys, 0, p.k, batch, row, kh, n, keys, p.wide);
            load_tile<T, kChunk, KD, kChainThreads>(tid, sm + Space::q, Space::kKeys, 0, p.q, batch, row, kh, n, keys, p.wide);
            if constexpr (kBack) {
                load_tile<T, kChunk, kMostValues, kChainThreads>(tid, sm + Space::v, Space::kValues, 0, bp.grad_out, batch,
                                                                        row, head, n, p.values, p.wide);
            } else {
                const T *src = delta_at<T>(p.v, batch, row, head);
                constexpr int kEach = 16 / int(sizeof(T)), kRow = kMostValues / kEach;
#pragma unroll 4
                for (int e = tid; e < kChunk * kRow; e += kChainThreads) {
                    const int i = e / kRow, j = e % kRow * kEach, left = i < n ? p.values - j : 0;
                    T *to = reinterpret_cast<T *>(sm + Space::v) + i * kMostValues + j;
                    if (p.wide) {
                        copy16(smem_addr(to), left > 0 ? src + i * p.v.row + j : src, left > 0 ? 16u : 0u);
                    } else {
#pragma unroll
                        for (int l = 0; l < kEach; ++l) to[l] = l < left ? src[i * p.v.row + j + l] : from_f32<T>(0.0f);
                    }
                }
            }
            copies_done();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[0]);
        };
        // the state as the next products' operand, and as kept
        auto put_state = [&] {
#pragma unroll
            for (int k = 0; k < kH; k += 16) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) split2(S[k + 2 * j], S[k + 2 * j + 1], hi[j], lo[j]);
                tmem_store(mine + kS + (k0 + k) / 2, hi);
                tmem_store(mine + kS + KD / 2 + (k0 + k) / 2, lo);
                if (kept)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int key = k0 + k + j * 8;
                        char *to = sm + Space::keep + uint32_t(key / 64) * kMostValues * kTileRow +
                                   tile_piece(uint32_t(dv), uint32_t(key % 64 / 8));
                        *reinterpret_cast<uint4 *>(to) = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
                        *reinterpret_cast<uint4 *>(to + Space::kKeep / 2) =
                            make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
                    }
            }
            arrive(0);
        };
        float o1[kT];  // forward: what the state gives to the outputs
        T o[kT];       // forward: the outputs of the chunk before
        auto finish_out = [&](int step) {
            wait_done(4, step);
            float o2[kT];
            read(o2, kD1 + t0);
#pragma unroll
            for (int j = 0; j < kT; ++j) o[j] = from_f32<T>(fmaf(p.scale, o2[j], o1[j]));
        };
        auto put_out = [&](int step) {
            T *to = out_place(step) + t0 * kMostValues + dv;
#pragma unroll
            for (int j = 0; j < kT; ++j) to[j * kMostValues] = o[j];
        };
        // back: the queries' side, scale e^G dO, in two pieces
        uint32_t side_hi[kBack ? kT / 2 : 1], side_lo[kBack ? kT / 2 : 1];
        auto prepare_side = [&](int step) {
            const int st = stage_of(step);
            const char *dO = sm + st * Space::bytes + Space::v;
            wait(full[st], round_of(step), kChainSide);
            const float4 *const first4 = reinterpret_cast<const float4 *>(rows_of[st].first + t0);
#pragma unroll
            for (int j = 0; j < kT; j += 4) {
                const float4 f = first4[j / 4];
                float x[4] = {p.scale * f.x, p.scale * f.y, p.scale * f.z, p.scale * f.w};
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    const char *e = dO + tile_at(uint32_t(t0 + j + l), uint32_t(dv), kChunk);
                    float d = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(e));
                    if constexpr (kP == 2) d += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(e + Space::kValues));
                    x[l] *= d;
                }
                split2(x[0], x[1], side_hi[kBack ? j / 2 : 0], side_lo[kBack ? j / 2 : 0]);
                split2(x[2], x[3], side_hi[kBack ? j / 2 + 1 : 0], side_lo[kBack ? j / 2 + 1 : 0]);
            }
        };
        if (chunks > 0) {
            put_state();
            if constexpr (!kMaps) load_rows(0);
            if constexpr (kBack) prepare_side(0);
        }
        for (int step = 0; step < chunks; ++step) {
            const int st = stage_of(step);
            char *s = sm + st * Space::bytes;
            const int64_t at = (slot0 + chunk_of(step)) * p.heads + head;
            if constexpr (!kBack)
                if (whole_part && step > 0) finish_out(step - 1);
            // what was put in shared memory last is copied on while the product runs
            if ((!kBack && whole_part) || kept) {
                meet();
                if (kept) copy_state(at);
                if (!kBack && step > 1) copy_out(step - 2);
            }
            // V's place in the stage of the chunk before: the outputs there are on their way
            if (Space::kOutInV && kept && step > 0) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[stage_of(step - 1)]);
            }
            wait(full[st], round_of(step), kChainRows);
            const ChainRows &r = rows_of[st];
            const float whole = r.first[kChunk - 1];
            const float4 *const first4 = reinterpret_cast<const float4 *>(r.first + t0);
            const float4 *const beta4 = reinterpret_cast<const float4 *>(r.beta + t0);
            const float4 *const rest4 = reinterpret_cast<const float4 *>(r.rest + t0);
            float x[kT];
            if constexpr (!kBack) {
                float y[kT];
                const T *v = reinterpret_cast<const T *>(s + Space::v) + t0 * kMostValues + dv;
#pragma unroll
                for (int j = 0; j < kT; ++j) y[j] = unit ? 0.0f : to_f32<T>(v[j * kMostValues]);
                wait_done(0, step);
                read(x, kD0 + t0);
#pragma unroll
                for (int j = 0; j < kT / 4; ++j) {
                    const float4 f = first4[j], b = beta4[j];
                    x[4 * j] = b.x * fmaf(-f.x, x[4 * j], y[4 * j]);
                    x[4 * j + 1] = b.y * fmaf(-f.y, x[4 * j + 1], y[4 * j + 1]);
                    x[4 * j + 2] = b.z * fmaf(-f.z, x[4 * j + 2], y[4 * j + 2]);
                    x[4 * j + 3] = b.w * fmaf(-f.w, x[4 * j + 3], y[4 * j + 3]);
                }
                put_rows(kR, x);
            } else {
                if constexpr (kBack) {
                    tmem_store(mine + kU + quarter * (kT / 2), side_hi);
                    tmem_store(mine + kU + 32 + quarter * (kT / 2), side_lo);
                }
                wait_done(0, step);
                read(x, kD0 + t0);
                wait_done(1, step);
                float y[kT] = {};
                if (!unit) read(y, kD1 + t0);
#pragma unroll
                for (int j = 0; j < kT / 4; ++j) {
                    const float4 f = rest4[j];
                    x[4 * j] = fmaf(f.x, x[4 * j], p.scale * y[4 * j]);
                    x[4 * j + 1] = fmaf(f.y, x[4 * j + 1], p.scale * y[4 * j + 1]);
                    x[4 * j + 2] = fmaf(f.z, x[4 * j + 2], p.scale * y[4 * j + 2]);
                    x[4 * j + 3] = fmaf(f.w, x[4 * j + 3], p.scale * y[4 * j + 3]);
                }
                put_rows(kR, x);
            }
            arrive(1);
            if (Space::kOutInV && !kept && lane == 0) mbar_arrive(&empty[st]);  // V has been read
            if ((!kBack && whole_part) || kept) meet();  // every copy has read its place
            if (!kBack && whole_part) {
                wait_done(1, step);
                read(o1, kDS + t0);
#pragma unroll
                for (int j = 0; j < kT / 4; ++j) {
                    const float4 f = first4[j];
                    o1[4 * j] *= p.scale * f.x, o1[4 * j + 1] *= p.scale * f.y;
                    o1[4 * j + 2] *= p.scale * f.z, o1[4 * j + 3] *= p.scale * f.w;
                }
            }
            wait_done(2, step);
            read(x, kD0 + t0);
            if (kept) {
#pragma unroll
                for (int j = 0; j < kT / 2; ++j) {
                    uint32_t hi, lo;
                    split2(x[2 * j], x[2 * j + 1], hi, lo);
                    char *a = sm + Space::keep + tile_at(uint32_t(t0 + 2 * j), uint32_t(dv), kChunk);
                    char *b = sm + Space::keep + tile_at(uint32_t(t0 + 2 * j + 1), uint32_t(dv), kChunk);
                    *reinterpret_cast<uint16_t *>(a) = uint16_t(hi), *reinterpret_cast<uint16_t *>(b) = uint16_t(hi >> 16);
                    *reinterpret_cast<uint16_t *>(a + Space::kValues) = uint16_t(lo);
                    *reinterpret_cast<uint16_t *>(b + Space::kValues) = uint16_t(lo >> 16);
                }
            }
            if constexpr (!kBack) put_rows(kU, x);
#pragma unroll
            for (int j = 0; j < kT / 4; ++j) {
                float4 f = kBack ? beta4[j] : rest4[j];
                if constexpr (kBack) {
                    const float4 e = first4[j];
                    f = make_float4(-f.x * e.x, -f.y * e.y, -f.z * e.z, -f.w * e.w);
                }
                x[4 * j] *= f.x, x[4 * j + 1] *= f.y, x[4 * j + 2] *= f.z, x[4 * j + 3] *= f.w;
            }
            put_rows(kR, x);
            arrive(2);
            // while the state's product runs
            if (kept) {
                meet();
                copy_rows(at);
            }
            if constexpr (!kBack) {
                if (whole_part && step > 0) put_out(step - 1);
            } else if (kStages == 2 && step + 1 < chunks) {
                prepare_side(step + 1);
            }
            wait_done(3, step);
#pragma unroll
            for (int k = 0; k < kH; k += kT) {
                read(x, kDS + k0 + k);
#pragma unroll
                for (int j = 0; j < kT; ++j) S[k + j] = fmaf(whole, S[k + j], x[j]);
            }
            if (step + 1 < chunks) {
                if (kept) meet();
                put_state();
                if constexpr (!kMaps) {
                    wait(empty[0], uint32_t(step), kChainRoom);
                    load_rows(step + 1);
                    if constexpr (kBack) prepare_side(step + 1);
                }
            }
        }
        if constexpr (!kBack)
            if (whole_part && chunks > 0) finish_out(chunks - 1);
        if (!all_well()) {
            in_vain = 1;
        } else {
            if (!kBack && whole_part && chunks > 0) {
                if (chunks > 1) copy_out(chunks - 2);
                meet();
                put_out(chunks - 1);
                meet();
                copy_out(chunks - 1);
            }
            float *to = walk.end_state(bp);
            if (to && dv < values) {
                to += dv;
#pragma unroll
                for (int k = 0; k < kH; ++k)
                    if (k0 + k < keys) to[int64_t(k0 + k) * values] = S[k];
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 0) tmem_free(tm, 512);
    if (in_vain) chain_give_up<T, KD, kBack, kPass>(bp);
}

template <class T, int KD, bool kBack, bool kMaps, int kPass>
cudaError_t chain_n(const DeltaBackwardParams &p, const DeltaMaps &maps, cudaStream_t s) {
    const auto kernel = delta_chain_kernel<T, KD, kBack, kMaps, kPass>;
    constexpr size_t bytes = ChainSpace<T, KD, kBack, kMaps>::kAll;
    constexpr int threads = kChainThreads + kHelpThreads;
    if (device_blocks(reinterpret_cast<const void *>(kernel), threads, bytes) == 0) return cudaErrorInvalidConfiguration;
    const uint32_t jobs = kPass == 0 ? 1u : uint32_t(kPass == 1 ? 2 * p.f.parts - 3 : p.f.parts - 1);
    return launch_pdl(kernel, dim3(uint32_t(p.f.sequences), uint32_t(p.f.heads), jobs), dim3(threads), bytes, s, p, maps);
}

template <class T, int KD, bool kBack>
cudaError_t chain_maps(const DeltaBackwardParams &p, const DeltaMaps &maps, int pass, cudaStream_t s) {
    if (pass == 0) return chain_n<T, KD, kBack, true, 0>(p, maps, s);
    return pass == 1 ? chain_n<T, KD, kBack, true, 1>(p, maps, s) : chain_n<T, KD, kBack, true, 2>(p, maps, s);
}

template <class T, bool kBack>
cudaError_t chain_t(const DeltaBackwardParams &p, const DeltaMaps &maps, int pass, cudaStream_t s) {
    const DeltaParams &f = p.f;
    if constexpr (kPieces<T> == 1)
        if (maps.made)
            return f.keys <= 64 ? chain_maps<T, 64, kBack>(p, maps, pass, s) : chain_maps<T, 128, kBack>(p, maps, pass, s);
    // others are not cut in parts: there is no pass but the one
    return f.keys <= 64 ? chain_n<T, 64, kBack, false, 0>(p, maps, s) : chain_n<T, 128, kBack, false, 0>(p, maps, s);
}

}  // namespace

}  // namespace dwp
