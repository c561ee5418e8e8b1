// Gated delta rule, the gradients of a chunk's rows, from the state before it,
// its corrections U, the gradient of the state after it and that of the
// corrections' right sides, dR:
//
//   dA = scale exp(G_i - G_j) dO_i.U_j (j <= i),  E = -exp(G_i - G_j) dR_i.U_j (j < i)
//   dQ = scale e^G dO S0^T + dA K
//   Z  = E K - e^G dR S0^T,   Y = e^{G_C - G} U dS1^T + dA^T Q + (beta E)^T K
//   dK = beta Z + Y,   dV = beta dR,   dbeta = dR.V + k.Z
//   dG = q.dQ + beta k.Z - k.Y, and <S1, dS1> at the chunk's last row; dg its
//   sum from the last row down
//
// (dG: G_i is in e^{G_i} q_i and, as e^{G_i} beta_i k_i and e^{-G_i} k_i, in
// what k_i does first and what it does to later rows.)
//
// A block has one chunk and key head and goes over the heads that share it,
// adding their dQ and dK in registers.  The products with the states and the
// second ones have the keys as rows and the chunk's rows as columns; dA and E
// come from one product of [dO; dR] with U.  Numbers that are not bf16 are in
// two pieces, and all four products of two such are taken; dA and E are in three,
// since the gradient of g is a sum of their products in which much cancels.
//
// 4 x 2048 rows x 16 heads of 128 x 128 take 264 us (239 with two pieces of dA
// and E and without the smallest products), of which moving the data is 93 (543
// MB read, 88 written): 2,048 blocks of one chunk each wait for their states and
// rows (long scoreboard 3.7 cycles an instruction, barriers 2.4; one block fits
// an SM), tensor cores are 14% busy.  Tried before that and slower than 239:
// asking for the next block's rows ahead of it (275), loads earlier in the block
// (273), blocks of one chunk's heads together (287), S1 through shared memory (246).
#pragma once

#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kGradThreads = 512;
constexpr int kMost = 128;  // keys and values, zeros past their own count
constexpr int kCols = 16;   // of the chunk's rows, a thread's share

template <class T>
struct GradSpace {
    static constexpr int kP = kPieces<T>;
    static constexpr uint32_t kRows = kChunk * kMost * 2, kState = kMost * kMost * 2;
    // keys and queries; [dO; dR] (hi, lo), later [dA; E] and beta E; U (hi, lo);
    // the state before the chunk, later the gradient of the one after it (hi, lo)
    static constexpr uint32_t k = 0, q = k + kP * kRows, stack = q + kP * kRows, u = stack + 4 * kRows;
    static constexpr uint32_t state = u + 2 * kRows, cross = stack, scaled = stack + 2 * kRows;
    // third pieces: of [dA; E], and for bf16 rows of beta E
    static constexpr uint32_t cross_third = scaled + kRows, scaled_third = state + 2 * kState;
    static constexpr uint32_t bytes = scaled_third + (kP == 1 ? kRows / 2 : 0);
    static constexpr size_t kAll = 1024 + bytes;
};

// Sums over the 32 lanes of each of 32 numbers: lane l gets that of number l.
__device__ __forceinline__ float sums_of_32(float (&x)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float give = up ? x[j] : x[j + o], keep = up ? x[j + o] : x[j];
            x[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    return x[0];
}

__device__ __forceinline__ float2 pair_of(uint32_t hi, uint32_t lo) {
    return make_float2(__uint_as_float(hi << 16) + __uint_as_float(lo << 16),
                       __uint_as_float(hi & 0xffff0000u) + __uint_as_float(lo & 0xffff0000u));
}

// Eight numbers in three pieces of bf16.
__device__ __forceinline__ void store_thirds(char *hi, char *lo, char *third, uint32_t at, const float (&f)[8]) {
    uint32_t h[4], l[4], t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        split2(f[2 * j], f[2 * j + 1], h[j], l[j]);
        const float2 two = pair_of(h[j], l[j]);
        const __nv_bfloat162 rest = __floats2bfloat162_rn(f[2 * j] - two.x, f[2 * j + 1] - two.y);
        t[j] = *reinterpret_cast<const uint32_t *>(&rest);
    }
    *reinterpret_cast<uint4 *>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    if (third) *reinterpret_cast<uint4 *>(third + at) = make_uint4(t[0], t[1], t[2], t[3]);
}

// kMaps: bf16 rows of whole 16-byte pieces, which come by tensor maps.
template <class T, bool kMaps>
__global__ void __launch_bounds__(kGradThreads, 1)
    delta_grad_kernel(DeltaBackwardParams bp, const __grid_constant__ DeltaMaps maps) {
    using Space = GradSpace<T>;
    constexpr int kP = Space::kP;
    constexpr uint32_t kRows = Space::kRows, kState = Space::kState, kTileBytes = kChunk * kTileRow;
    extern __shared__ char raw[];
    __shared__ Sum2 sums[kChunk];
    __shared__ float beta[kChunk], first[kChunk], rest[kChunk], value_dot[kChunk];
    __shared__ uint64_t bars[5], drained;
    __shared__ uint32_t tmem;
    const DeltaParams &p = bp.f;
    char *sm = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
    // sums over the keys, in U's place when its products have ended
    struct Dots {
        float key[4][kChunk], all[4][kChunk], whole[kGradThreads / 32];
    };
    Dots &dots = *reinterpret_cast<Dots *>(sm + Space::u);
    pdl_trigger();
    pdl_wait();
    const DeltaChunk c = delta_chunk(p, blockIdx.x);
    if (c.rows == 0) return;
    const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
    const int part = warp / 4, dk = warp % 4 * 32 + lane, t0 = part * kCols, n = c.rows;
    const int kh = blockIdx.y, per = p.heads / p.key_heads, keys = p.keys, values = p.values;
    const int tiles = (keys + 63) / 64, value_tiles = (values + 63) / 64;
#ifdef DWP_DELTA_TEST
    __shared__ uint64_t never;
    if (tid == 0) mbar_init(&never, 1);
    Stall stall{&never, p.stall_site, p.stall_skip};
#endif
    if (tid == 0) {
        for (int i = 0; i < 5; ++i) mbar_init(&bars[i], 1);
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem, 512);
    // what no input fills: of the states' tiles, of the stack's, U's and the
    // second pieces of bf16 gradients
    for (int e = tid; e < 2 * kMost * kMost / 8; e += kGradThreads)
        if (e / 8 % kMost >= values || e / (kMost * 8) % 2 >= tiles)
            *reinterpret_cast<uint4 *>(sm + Space::state + uint32_t(e) * 16) = make_uint4(0, 0, 0, 0);
    if (value_tiles == 1)
        for (int e = tid; e < kChunk * 8; e += kGradThreads)
#pragma unroll
            for (int piece = 0; piece < 2; ++piece) {
                *reinterpret_cast<uint4 *>(sm + Space::u + piece * kRows + kTileBytes + e * 16) = make_uint4(0, 0, 0, 0);
            }
    fence_proxy_async_smem();
    __syncthreads();
    const uint32_t tm = tmem, mine = tm + (uint32_t(warp % 4) << 21);
    constexpr uint32_t kDX = 0, kDA = 128, kDW = 192, kDY = 320, kDU = 384;
    bool ok = true;  // no wait was in vain: of this thread, and, where they meet, of any
    auto read = [&](float (&x)[kCols], uint32_t at) {
        uint32_t v[kCols];
        tmem_load(v, mine + at);
        tmem_ready();
#pragma unroll
        for (int j = 0; j < kCols; ++j) x[j] = __uint_as_float(v[j]);
    };
    auto meet = [&] {
        copies_done();
        fence_proxy_async_smem();
        tmem_fence_before();
        ok = __syncthreads_and(ok);
        tmem_fence_after();
    };
    // a key's or query's entry `dk` of row i
    auto entry = [&](uint32_t tile, int i) {
        const char *at = sm + tile + tile_at(uint32_t(i), uint32_t(dk), kChunk);
        float f = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(at));
        if constexpr (kP == 2) f += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(at + kRows));
        return f;
    };
    // rows of zeros where the chunk is short (a map's box goes on into the next sequence)
    auto clear = [&](uint32_t tile, uint32_t tile_bytes, int first_row) {
        for (int e = tid; e < 2 * (kChunk - n) * 8; e += kGradThreads) {
            const int x = e / ((kChunk - n) * 8), l = e % ((kChunk - n) * 8);
            *reinterpret_cast<uint4 *>(sm + tile + x * tile_bytes + (first_row + n) * kTileRow + l * 16) = make_uint4(0, 0, 0, 0);
        }
    };
    float dq[kCols], dkey[kCols];
    int asked = 0;  // heads whose copies were issued, by thread 0
    for (int h = 0; h < per; ++h) {
        const int head = kh * per + h;
        const int64_t at = int64_t(blockIdx.x) * p.heads + head;
        const uint32_t parity = uint32_t(h & 1);
        auto wait = [&](int bar) {
#ifdef DWP_DELTA_TEST
            if (ok && stall.at(kGradFirst + bar)) ok = false;
#endif
            if (ok) ok = mma_wait(&bars[bar], parity);
            tmem_fence_after();
        };
        const char *S0 = reinterpret_cast<const char *>(p.states + at * tiles * 64 * values);
        const char *S1 = reinterpret_cast<const char *>(bp.ends + at * tiles * 64 * values);
        const char *kept_u = reinterpret_cast<const char *>(p.u + at * value_tiles * 64 * kChunk);
        const char *kept_dr = reinterpret_cast<const char *>(bp.dr + at * value_tiles * 64 * kChunk);
        // where the last head's [dA; E] were, zeros again
        if constexpr (kP == 1)
            for (int e = tid; e < 2 * kChunk * 8; e += kGradThreads)
                *reinterpret_cast<uint4 *>(sm + Space::stack + 2 * kRows + e / (kChunk * 8) * 2 * kTileBytes +
                                           e % (kChunk * 8) * 16) = make_uint4(0, 0, 0, 0);
        if (value_tiles == 1)
            for (int e = tid; e < kChunk * 8; e += kGradThreads)
#pragma unroll
                for (int piece = 0; piece < 2; ++piece)
                    *reinterpret_cast<uint4 *>(sm + Space::stack + piece * 2 * kRows + 3 * kTileBytes + e * 16) =
                        make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0 && ok) {
            ++asked;
            const uint32_t each = uint32_t(values) * kTileRow;
            mbar_arrive_expect_tx(&bars[3], 2 * tiles * each + 4 * value_tiles * kTileBytes +
                                                (kMaps ? 2 * kTileBytes + (h == 0 ? 4 * kTileBytes : 0) : 0));
            if constexpr (kMaps) {
                const int r = int(c.row), b = int(c.batch);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    map_load(sm + Space::stack + x * 2 * kTileBytes, &maps.v, &bars[3], x * 64, head, r, b);
                    if (h == 0) {
                        map_load(sm + Space::k + x * kTileBytes, &maps.k, &bars[3], x * 64, kh, r, b);
                        map_load(sm + Space::q + x * kTileBytes, &maps.q, &bars[3], x * 64, kh, r, b);
                    }
                }
            }
            for (int piece = 0; piece < 2; ++piece) {
                for (int i = 0; i < value_tiles; ++i)
                    bulk_load(sm + Space::stack + piece * 2 * kRows + i * 2 * kTileBytes + kTileBytes,
                              kept_dr + (piece * value_tiles + i) * kTileBytes, kTileBytes, &bars[3]);
                bulk_load(sm + Space::u + piece * kRows, kept_u + piece * value_tiles * kTileBytes, value_tiles * kTileBytes,
                          &bars[3]);
                for (int i = 0; i < tiles; ++i)
                    bulk_load(sm + Space::state + piece * kState + i * kMost * kTileRow, S0 + int64_t(piece * tiles + i) * each,
                              each, &bars[3]);
            }
        }
        if constexpr (!kMaps) {
            if (h == 0) {
                load_tile<T, kChunk, kMost, kGradThreads>(tid, sm + Space::k, kRows, 0, p.k, c.batch, c.row, kh, n, keys, p.wide);
                load_tile<T, kChunk, kMost, kGradThreads>(tid, sm + Space::q, kRows, 0, p.q, c.batch, c.row, kh, n, keys, p.wide);
            }
            load_tile<T, 2 * kChunk, kMost, kGradThreads>(tid, sm + Space::stack, 2 * kRows, 0, bp.grad_out, c.batch, c.row,
                                                                 head, n, values, p.wide);
        }
        // this thread's values of V: two pieces of eight
        float v[2][8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = e * (kGradThreads / 16) + tid / 16, j0 = tid % 16 * 8;
            const int left = i < n ? values - j0 : 0;
            const T *from = delta_at<T>(p.v, c.batch, c.row + (i < n ? i : 0), head) + (left > 0 ? j0 : 0);
            if (p.wide) load_eight<T, true>(v[e], from, left);
            else load_eight<T, false>(v[e], from, left);
        }
        if (warp == 15) {
            float g[2];
            Sum2 s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane + 32 * i;
                g[i] = r < n ? delta_g(p.g, c.batch, c.row + r, head) : 0.0f;
                beta[r] = r < n ? delta_beta<T>(p, c.batch, c.row + r, head) : 0.0f;
            }
            delta_sums(s, g);
            const Sum2 last = {__shfl_sync(0xffffffffu, s[1].hi, 31), __shfl_sync(0xffffffffu, s[1].lo, 31)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float e = __expf(s[i].hi);
                sums[lane + 32 * i] = s[i];
                first[lane + 32 * i] = fmaf(e, s[i].lo, e);
                rest[lane + 32 * i] = __expf(sum2_less(last, s[i]));
            }
        }
        wait(3);
        if (kMaps && n < kChunk) {
            clear(Space::stack, 2 * kTileBytes, 0);
            if (h == 0) clear(Space::k, kTileBytes, 0), clear(Space::q, kTileBytes, 0);
        }
        meet();
        const Operand<kChunk, false> U(sm + Space::u), Ul(sm + Space::u + kRows);
        const Operand<kMost, true> S(sm + Space::state), Sl(sm + Space::state + kState);
        if (warp == 0 && elect_one() && ok) {
            const Operand<2 * kChunk, false> both(sm + Space::stack), bothl(sm + Space::stack + 2 * kRows);
            product_ss<kChunk, kMost>(tm + kDA, both, U, false);
            product_ss<kChunk, kMost>(tm + kDA, both, Ul, true);
            product_ss<kChunk, kMost>(tm + kDA, bothl, U, true);
            product_ss<kChunk, kMost>(tm + kDA, bothl, Ul, true);
            mma_commit(&bars[0]);
            product_ss<2 * kChunk, kMost>(tm + kDX, S, both, false);
            product_ss<2 * kChunk, kMost>(tm + kDX, Sl, both, true);
            if constexpr (kP == 2) {
                product_ss<2 * kChunk, kMost>(tm + kDX, S, bothl, true);
                product_ss<2 * kChunk, kMost>(tm + kDX, Sl, bothl, true);
            } else {
                const Operand<2 * kChunk, false> drl(sm + Space::stack + 2 * kRows + kTileBytes);
                product_ss<kChunk, kMost>(tm + kDX + kChunk, S, drl, true);
                product_ss<kChunk, kMost>(tm + kDX + kChunk, Sl, drl, true);
            }
            mma_commit(&bars[1]);
        }
        // the gradient of the state after the chunk, on its way into registers
        uint4 ends[4][2];
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            const int e = tid + l * kGradThreads;
            ends[l][0] = ends[l][1] = make_uint4(0, 0, 0, 0);
            if (e < tiles * values * 8) {
                ends[l][0] = *reinterpret_cast<const uint4 *>(S1 + e * 16);
                ends[l][1] = *reinterpret_cast<const uint4 *>(S1 + (tiles * values * 8 + e) * 16);
            }
        }
        // dV, and dR.V
        const float in_vain = ok ? 0.0f : not_a_number();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = e * (kGradThreads / 16) + tid / 16, j0 = tid % 16 * 8, left = values - j0;
            const char *from = sm + Space::stack + j0 / 64 * 2 * kTileBytes + tile_piece(uint32_t(kChunk + i), uint32_t(j0 % 64 / 8));
            const uint4 hi = *reinterpret_cast<const uint4 *>(from), lo = *reinterpret_cast<const uint4 *>(from + 2 * kRows);
            const float2 f[4] = {pair_of(hi.x, lo.x), pair_of(hi.y, lo.y), pair_of(hi.z, lo.z), pair_of(hi.w, lo.w)};
            float s = 0.0f, d[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s = fmaf(f[j].x, v[e][2 * j], fmaf(f[j].y, v[e][2 * j + 1], s));
                d[2 * j] = fmaf(beta[i], f[j].x, in_vain), d[2 * j + 1] = fmaf(beta[i], f[j].y, in_vain);
            }
            if (i < n && left > 0) {
                T *to = delta_at<T>(bp.grad_v, c.batch, c.row + i, head) + j0;
                // dense rows of whole 16-byte pieces start on 16 bytes if the first does
                if (p.wide && bp.wide && left >= 8) {
                    store_f32<8>(to, d);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < left) to[j] = from_f32<T>(d[j]);
                }
            }
#pragma unroll
            for (int o = 8; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane % 16 == 0) value_dot[i] = s;
        }
        // dA and E: this thread's row, and a quarter of the columns
        float w[kCols];
        wait(0);
        read(w, kDA + t0);
        const int row = dk % kChunk;
        const bool cross = dk >= kChunk;
        {
            const Sum2 own = sums[row];
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const int col = t0 + j;
                const bool in = cross ? col < row : col <= row;
                w[j] = in ? (cross ? -1.0f : p.scale) * __expf(sum2_less(own, sums[col])) * w[j] : 0.0f;
            }
        }
        wait(1);
        __syncthreads();  // the stack and the state have been read, by products and threads
#pragma unroll
        for (int j = 0; j < kCols / 8; ++j) {
            float f[8];
#pragma unroll
            for (int l = 0; l < 8; ++l) f[l] = w[j * 8 + l];
            const uint32_t piece = uint32_t(t0 / 8 + j);
            store_thirds(sm + Space::cross, sm + Space::cross + kRows, sm + Space::cross_third, tile_piece(uint32_t(dk), piece), f);
            if (cross) {
#pragma unroll
                for (int l = 0; l < 8; ++l) f[l] *= beta[row];
                store_thirds(sm + Space::scaled, sm + Space::scaled + kTileBytes, kP == 1 ? sm + Space::scaled_third : nullptr,
                             tile_piece(uint32_t(row), piece), f);
            }
        }
        // the gradient of the state after the chunk takes the state's place, and meets it on the way
        float meeting = 0.0f;
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            const int e = tid + l * kGradThreads;
            if (e >= tiles * values * 8) continue;
            uint4 *at_hi = reinterpret_cast<uint4 *>(sm + Space::state + (e >= values * 8 ? kMost * 8 + e - values * 8 : e) * 16);
            uint4 *at_lo = reinterpret_cast<uint4 *>(reinterpret_cast<char *>(at_hi) + kState);
            const uint4 shi = *at_hi, slo = *at_lo;
            auto with = [&](uint32_t a, uint32_t b, uint32_t x, uint32_t y) {
                const float2 f = pair_of(a, b), g = pair_of(x, y);
                meeting = fmaf(f.x, g.x, fmaf(f.y, g.y, meeting));
            };
            with(ends[l][0].x, ends[l][1].x, shi.x, slo.x), with(ends[l][0].y, ends[l][1].y, shi.y, slo.y);
            with(ends[l][0].z, ends[l][1].z, shi.z, slo.z), with(ends[l][0].w, ends[l][1].w, shi.w, slo.w);
            *at_hi = ends[l][0], *at_lo = ends[l][1];
        }
        meeting *= first[kChunk - 1];
        meet();
        if (warp == 0 && elect_one() && ok) {
            const Operand<kChunk, true> K(sm + Space::k), Q(sm + Space::q);
            const Operand<2 * kChunk, false> W(sm + Space::cross), Wl(sm + Space::cross + kRows);
            const Operand<2 * kChunk, true> A(sm + Space::cross), Al(sm + Space::cross + kRows);
            const Operand<kChunk, true> E(sm + Space::scaled), El(sm + Space::scaled + kTileBytes);
            product_ss<2 * kChunk, kChunk>(tm + kDW, K, W, false);
            product_ss<2 * kChunk, kChunk>(tm + kDW, K, Wl, true);
            product_ss<kChunk, kChunk>(tm + kDY, Q, A, false);
            product_ss<kChunk, kChunk>(tm + kDY, Q, Al, true);
            product_ss<kChunk, kChunk>(tm + kDY, K, E, true);
            product_ss<kChunk, kChunk>(tm + kDY, K, El, true);
            product_ss<2 * kChunk, kChunk>(tm + kDW, K, Operand<2 * kChunk, false>(sm + Space::cross_third), true);
            product_ss<kChunk, kChunk>(tm + kDY, Q, Operand<2 * kChunk, true>(sm + Space::cross_third), true);
            if constexpr (kP == 1) {
                product_ss<kChunk, kChunk>(tm + kDY, K, Operand<kChunk, true>(sm + Space::scaled_third), true);
            } else {
                const Operand<kChunk, true> Kl(sm + Space::k + kRows), Ql(sm + Space::q + kRows);
                product_ss<2 * kChunk, kChunk>(tm + kDW, Kl, W, true);
                product_ss<2 * kChunk, kChunk>(tm + kDW, Kl, Wl, true);
                product_ss<kChunk, kChunk>(tm + kDY, Ql, A, true);
                product_ss<kChunk, kChunk>(tm + kDY, Ql, Al, true);
                product_ss<kChunk, kChunk>(tm + kDY, Kl, E, true);
                product_ss<kChunk, kChunk>(tm + kDY, Kl, El, true);
            }
            mma_commit(&bars[2]);
            product_ss<kChunk, kMost>(tm + kDU, S, U, false);
            product_ss<kChunk, kMost>(tm + kDU, S, Ul, true);
            product_ss<kChunk, kMost>(tm + kDU, Sl, U, true);
            product_ss<kChunk, kMost>(tm + kDU, Sl, Ul, true);
            mma_commit(&bars[4]);
        }
        float x[kCols], both_sums[2 * kCols];  // of q.dQ + beta k.Z - k.Y, and of k.Z
        wait(2);
        // dQ
        read(w, kDX + t0);
        read(x, kDW + t0);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const float d = fmaf(p.scale * first[t0 + j], w[j], x[j]);
            dq[j] = h ? dq[j] + d : d;
            both_sums[j] = d * entry(Space::q, t0 + j);
        }
        // Z
        read(w, kDX + kChunk + t0);
        read(x, kDW + kChunk + t0);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const float z = fmaf(-first[t0 + j], w[j], x[j]), b = beta[t0 + j] * z, k = entry(Space::k, t0 + j);
            dkey[j] = h ? dkey[j] + b : b;
            both_sums[kCols + j] = k * z;
            both_sums[j] = fmaf(k, b, both_sums[j]);
        }
        // Y
        read(x, kDY + t0);
        wait(4);
        read(w, kDU + t0);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const float r = rest[t0 + j] * w[j], y = r + x[j], k = entry(Space::k, t0 + j);
            meeting = fmaf(k, r, meeting);
            dkey[j] += y;
            both_sums[j] = fmaf(-k, y, both_sums[j]);
        }
        const float sum = sums_of_32(both_sums, lane);
        if (lane < kCols) dots.all[warp % 4][t0 + lane] = sum;
        else dots.key[warp % 4][t0 + lane - kCols] = sum;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) meeting += __shfl_xor_sync(0xffffffffu, meeting, o);
        if (lane == 0) dots.whole[warp] = meeting;
        tmem_fence_before();
        ok = __syncthreads_and(ok);
        if (warp == 15) {
            float whole = 0.0f;
            for (int w = 0; w < kGradThreads / 32; ++w) whole += dots.whole[w];
            const float bad = ok ? 0.0f : not_a_number();
            float g[2];
            Sum2 sum[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = kChunk - 1 - (lane + 32 * r);
                g[r] = i >= n ? 0.0f : (dots.all[0][i] + dots.all[1][i]) + (dots.all[2][i] + dots.all[3][i]) +
                                           (i == n - 1 ? whole : 0.0f) + bad;
            }
            delta_sums(sum, g);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = kChunk - 1 - (lane + 32 * r);
                if (i >= n) continue;
                if (bp.grad_g.data) *delta_at<float>(bp.grad_g, c.batch, c.row + i, head) = sum[r].hi;
                const float d = value_dot[i] + ((dots.key[0][i] + dots.key[1][i]) + (dots.key[2][i] + dots.key[3][i])) + bad;
                if (p.beta_f32) *delta_at<float>(bp.grad_beta, c.batch, c.row + i, head) = d;
                else *delta_at<T>(bp.grad_beta, c.batch, c.row + i, head) = from_f32<T>(d);
            }
        }
    }
    if (dk < keys) {
        T *to_q = delta_at<T>(bp.grad_q, c.batch, c.row + t0, kh) + dk, *to_k = delta_at<T>(bp.grad_k, c.batch, c.row + t0, kh) + dk;
        const float bad = ok ? 0.0f : not_a_number();
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (t0 + j < n) {
                to_q[j * bp.grad_q.row] = from_f32<T>(dq[j] + bad);
                to_k[j * bp.grad_k.row] = from_f32<T>(dkey[j] + bad);
            }
    }
    __syncthreads();
    if (warp == 0) {
        if (!ok) {
            if (asked > 0) mma_wait(&bars[3], uint32_t(asked - 1) & 1u);
            __syncwarp();
            if (elect_one()) mma_commit(&drained);
            mma_wait(&drained, 0);
        }
        __syncwarp();
        tmem_free(tm, 512);
    }
}

template <class T, bool kMaps>
cudaError_t grad_k(const DeltaBackwardParams &p, const DeltaMaps &maps, cudaStream_t s) {
    const auto kernel = delta_grad_kernel<T, kMaps>;
    constexpr size_t bytes = GradSpace<T>::kAll;
    if (device_blocks(reinterpret_cast<const void *>(kernel), kGradThreads, bytes) == 0) return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, dim3(uint32_t(p.f.slots), uint32_t(p.f.key_heads)), dim3(kGradThreads), bytes, s, p, maps);
}

template <class T>
cudaError_t grad_t(const DeltaBackwardParams &p, const DeltaMaps &maps, cudaStream_t s) {
    if constexpr (kPieces<T> == 1)
        if (maps.made) return grad_k<T, true>(p, maps, s);
    return grad_k<T, false>(p, maps, s);
}

}  // namespace

}  // namespace dwp
