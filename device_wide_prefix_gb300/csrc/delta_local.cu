// Gated delta rule, what a chunk needs of itself alone: the inverse
// T = (1 + L)^-1, L the strictly lower part of diag(beta) M, and the weights A,
// each in two planes of bf16.
//
// One product of [K; Q] with K gives k_i.k_j in the lanes of the first 64 rows
// and q_i.k_j in the others, for all heads that share the keys; teams of 128
// threads take the heads in turn.  A thread has one row; the rows of L go to
// shared memory.  The inverse is that of the four diagonal blocks of 16, by
// substitution with a thread a column, and then, of 16 and of 32,
// -T22 L21 T11 below each pair: the substitution's steps wait for one another.
// The loops are short on purpose: unrolled, three of ten cycles of a warp went
// to fetching instructions.
//
// 4 x 2048 rows, 16 key heads and 32 heads of 128 keys take 78 us, of which moving
// the data (201 MB) would be 30; 16 heads 45.  The substitutions' steps bound it:
// barriers are the longest wait (2.5 cycles an instruction), the scheduler issues
// 0.43 a cycle, tensor cores are 2% busy.
#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kTeam = 128;
constexpr int kPitch = kChunk + 4;  // words a row of L and T: rows start on 16 bytes, in other banks

template <class T, int KD, int kTeams>
constexpr size_t local_bytes = 1024 + size_t(kPieces<T>) * 2 * kChunk * KD * 2 + size_t(kTeams) * kChunk * kPitch * 4;

// kMaps: bf16 rows of whole 16-byte pieces, which come by tensor maps.  (Rows
// past a short chunk's are another sequence's: nothing that is kept reads them.)
template <class T, int KD, bool kMaps, int kTeams>
__global__ void __launch_bounds__(kTeam * kTeams, 4 / kTeams)
    delta_local_kernel(DeltaParams p, const __grid_constant__ DeltaMaps maps) {
    extern __shared__ char raw[];
    __shared__ Sum2 sums_[kTeams][kChunk];
    __shared__ float beta_[kTeams][kChunk];
    __shared__ uint64_t bar, landed;
    __shared__ uint32_t tmem;
    constexpr uint32_t kLo = 2 * kChunk * KD * 2;
    char *tile = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
    pdl_trigger();
    pdl_wait();
    const DeltaChunk c = delta_chunk(p, blockIdx.x);
    if (c.rows == 0) return;
    const int lane = threadIdx.x % 32, warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);
    const int team = warp / 4, in_team = warp % 4, tid = threadIdx.x % kTeam;
    const int kh = blockIdx.y, per = p.heads / p.key_heads;
    float *L = reinterpret_cast<float *>(tile + kPieces<T> * kLo) + team * kChunk * kPitch;  // and T, block by block
    Sum2 *sums = sums_[team];
    float *beta = beta_[team];
    auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(kTeam) : "memory"); };
#ifdef DWP_DELTA_TEST
    __shared__ uint64_t never;
    if (threadIdx.x == 0) mbar_init(&never, 1);
    Stall stall{&never, p.stall_site, p.stall_skip};
#endif
    auto wait = [&](uint64_t &b, [[maybe_unused]] WaitSite site) {
#ifdef DWP_DELTA_TEST
        if (stall.at(site)) return false;
#endif
        return mma_wait(&b, 0);
    };
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        mbar_init(&landed, 1);
        fence_mbar_init();
        if constexpr (kMaps) {
            mbar_arrive_expect_tx(&landed, kLo);
#pragma unroll
            for (int x = 0; x < KD; x += 64) {
                map_load(tile + 2 * x * kTileRow, &maps.k, &landed, x, kh, int(c.row), int(c.batch));
                map_load(tile + (2 * x + kChunk) * kTileRow, &maps.q, &landed, x, kh, int(c.row), int(c.batch));
            }
        }
    }
    // a head's log decays, and betas, by the team's first and last warp
    float g[2], b[2];
    auto load_rows = [&](int h) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = lane + 32 * i;
            const bool in = r < c.rows && h < per;
            if (in_team == 0) g[i] = in ? delta_g(p.g, c.batch, c.row + r, kh * per + h) : 0.0f;
            if (in_team == 3) b[i] = in ? delta_beta<T>(p, c.batch, c.row + r, kh * per + h) : 0.0f;
        }
    };
    load_rows(team);
    if constexpr (!kMaps) {
        load_tile<T, 2 * kChunk, KD, kTeam * kTeams>(threadIdx.x, tile, kLo, 0, p.k, c.batch, c.row, kh, c.rows, p.keys, p.wide);
        load_tile<T, 2 * kChunk, KD, kTeam * kTeams>(threadIdx.x, tile, kLo, kChunk, p.q, c.batch, c.row, kh, c.rows, p.keys,
                                                            p.wide);
        copies_done();
        fence_proxy_async_smem();
    }
    if (warp == 0) tmem_alloc(&tmem, kChunk);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t d = tmem;
    bool issued = false;
    if (warp == 0) {
        const bool rows_here = !kMaps || wait(landed, kLocalRows);
        __syncwarp();
        if (elect_one() && rows_here) {
            const Operand<2 * kChunk, false> hi(tile), lo(tile + kLo);
            product_ss<kChunk, KD>(d, hi, hi, false);
            if constexpr (kPieces<T> == 2) {
                product_ss<kChunk, KD>(d, hi, lo, true);
                product_ss<kChunk, KD>(d, lo, hi, true);
                product_ss<kChunk, KD>(d, lo, lo, true);
            }
            mma_commit(&bar);
            issued = true;
        }
        __syncwarp();
    }
    bool ok = true;
    const int row = tid % kChunk;  // of the chunk, as key or as query
    for (int h = team; h < per; h += kTeams) {
        const int64_t at = int64_t(blockIdx.x) * p.heads + kh * per + h;
        char *T_out = reinterpret_cast<char *>(p.inverse + at * kChunk * kChunk);
        char *A_out = reinterpret_cast<char *>(p.weights + at * kChunk * kChunk);
        sync();
        if (in_team == 0) {
            Sum2 s[2];
            delta_sums(s, g);
            sums[lane] = s[0], sums[lane + 32] = s[1];
        }
        if (in_team == 3) beta[lane] = b[0], beta[lane + 32] = b[1];
        load_rows(h + kTeams);
        sync();
        if (h == team) {
            ok = wait(bar, kLocalProduct);
            __syncwarp();
            tmem_fence_after();
        }
        const Sum2 mine = sums[row];
        const float scale = !ok ? not_a_number() : tid < kChunk ? beta[row] : 1.0f;
        // columns that this row reads: those before it, and a query's own
        const int cols = row < c.rows ? row + (tid >= kChunk) : 0;
#pragma unroll 1
        for (int j0 = 0; j0 < kChunk; j0 += 16) {
            float f[16] = {};
            if (j0 < row / 32 * 32 + 32) {  // the whole warp's
                uint32_t v[16];
                tmem_load(v, d + (uint32_t(in_team) << 21) + j0);
                tmem_ready();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float e = scale * __expf(sum2_less(mine, sums[j0 + j])) * __uint_as_float(v[j]);
                    f[j] = j0 + j < cols ? e : 0.0f;
                }
            }
            if (tid < kChunk) {
                float4 *to = reinterpret_cast<float4 *>(L + row * kPitch + j0);
#pragma unroll
                for (int j = 0; j < 4; ++j) to[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float e[8];
#pragma unroll
                    for (int l = 0; l < 8; ++l) e[l] = f[8 * j + l];
                    store_pieces(A_out, A_out + kChunk * kTileRow, tile_piece(uint32_t(row), uint32_t(j0 / 8 + j)), e);
                }
            }
        }
        sync();
        // the diagonal blocks' inverses: a thread has a column, in registers, then in the block's place
        if (in_team < 2) {
            const int block = in_team * 2 + lane / 16, col = lane % 16;
            float *B = L + block * 16 * (kPitch + 1);
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s[4] = {i == col ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(B + i * kPitch + j);
                    s[0] = fmaf(-l.x, x[j], s[0]);
                    if (j + 1 < i) s[1] = fmaf(-l.y, x[j + 1], s[1]);
                    if (j + 2 < i) s[2] = fmaf(-l.z, x[j + 2], s[2]);
                    if (j + 3 < i) s[3] = fmaf(-l.w, x[j + 3], s[3]);
                }
                x[i] = (s[0] + s[1]) + (s[2] + s[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) B[i * kPitch + col] = x[i];
        }
        sync();
        // below each pair of blocks of 16: first L21 T11 (into the unused upper
        // right), then -T22 of it in L21's place; a thread has four of a row
        {
            const int r = tid % 64 / 4, c0 = tid % 4 * 4, pair = tid / 64;
            float *top = L + pair * 32 * (kPitch + 1);  // T11; T22 16 rows and columns on
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                const float *a = top + (16 + r) * kPitch + (pass ? 16 : 0), *from = top + (pass ? 16 : 0) + c0;
                float s[4] = {};
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    const float4 x4 = *reinterpret_cast<const float4 *>(a + k);
                    const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int l = 0; l < 4; ++l) {
                        const float4 y = *reinterpret_cast<const float4 *>(from + (k + l) * kPitch);
                        s[0] = fmaf(x[l], y.x, s[0]), s[1] = fmaf(x[l], y.y, s[1]);
                        s[2] = fmaf(x[l], y.z, s[2]), s[3] = fmaf(x[l], y.w, s[3]);
                    }
                }
                float4 *to = reinterpret_cast<float4 *>(top + (pass ? 16 + r : r) * kPitch + (pass ? 0 : 16) + c0);
                to[0] = pass ? make_float4(-s[0], -s[1], -s[2], -s[3]) : make_float4(s[0], s[1], s[2], s[3]);
                sync();
            }
        }
        // the same below the blocks of 32; T11 and T22 are lower triangular, and a
        // warp leaves out what is zero (or, in their upper right, left from before)
        {
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                const int r = pass ? in_team * 8 + lane / 4 : lane, c0 = (pass ? lane % 4 : in_team) * 8;
                const float *a = L + (32 + r) * kPitch + (pass ? 32 : 0), *from = L + (pass ? 32 : 0) + c0;
                const int first = pass ? 0 : c0, last = pass ? in_team * 8 + 8 : 32;
                float s[8] = {};
#pragma unroll 1
                for (int k = first; k < last; k += 4) {
                    const float4 x4 = *reinterpret_cast<const float4 *>(a + k);
                    const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int l = 0; l < 4; ++l) {
                        const float4 y0 = *reinterpret_cast<const float4 *>(from + (k + l) * kPitch);
                        const float4 y1 = *reinterpret_cast<const float4 *>(from + (k + l) * kPitch + 4);
                        s[0] = fmaf(x[l], y0.x, s[0]), s[1] = fmaf(x[l], y0.y, s[1]);
                        s[2] = fmaf(x[l], y0.z, s[2]), s[3] = fmaf(x[l], y0.w, s[3]);
                        s[4] = fmaf(x[l], y1.x, s[4]), s[5] = fmaf(x[l], y1.y, s[5]);
                        s[6] = fmaf(x[l], y1.z, s[6]), s[7] = fmaf(x[l], y1.w, s[7]);
                    }
                }
                float4 *to = reinterpret_cast<float4 *>(L + (pass ? 32 + r : r) * kPitch + (pass ? 0 : 32) + c0);
                to[0] = pass ? make_float4(-s[0], -s[1], -s[2], -s[3]) : make_float4(s[0], s[1], s[2], s[3]);
                to[1] = pass ? make_float4(-s[4], -s[5], -s[6], -s[7]) : make_float4(s[4], s[5], s[6], s[7]);
                sync();
            }
        }
#pragma unroll 1
        for (int e = tid; e < kChunk * kChunk / 8; e += kTeam) {
            const int i = e / 8, j0 = e % 8 * 8;
            float f[8];
            load_f32<8>(f, L + i * kPitch + j0);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = i / 16 < j0 / 16 ? 0.0f : f[j];
            store_pieces(T_out, T_out + kChunk * kTileRow, tile_piece(uint32_t(i), uint32_t(j0 / 8)), f);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 0) {
        if (!ok) {
            if (kMaps) mma_wait(&landed, 0);
            if (issued) mma_wait(&bar, 0);
        }
        __syncwarp();
        tmem_free(d, kChunk);
    }
}

template <class T, int KD, bool kMaps, int kTeams>
cudaError_t local_n(const DeltaParams &p, const DeltaMaps &maps, cudaStream_t s) {
    const auto kernel = delta_local_kernel<T, KD, kMaps, kTeams>;
    constexpr size_t bytes = local_bytes<T, KD, kTeams>;
    if (device_blocks(reinterpret_cast<const void *>(kernel), kTeam * kTeams, bytes) == 0) return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, dim3(uint32_t(p.slots), uint32_t(p.key_heads)), dim3(kTeam * kTeams), bytes, s, p, maps);
}

// Two teams share a block's keys where heads do, unless there are blocks enough
// without, of rows that maps bring (others take more threads to load and split).
// A call with one team against two, 128 x 128, bf16: 4 x 2048 rows x 16 key heads
// 193 us against 201, 4 key heads 196 against 202, 1 key head (128 blocks) of 16
// heads 192 against 168, 512 rows x 2 key heads of 16 heads 74 against 61; off 16
// bytes, 4 x 2048 rows x 16 key heads, 549 against 459, in f32 490 against 429.
template <class T, int KD, bool kMaps>
cudaError_t local_k(const DeltaParams &p, const DeltaMaps &maps, cudaStream_t s) {
    const bool many = kMaps && p.slots * p.key_heads > 3 * kSMs;
    return p.heads == p.key_heads || many ? local_n<T, KD, kMaps, 1>(p, maps, s) : local_n<T, KD, kMaps, 2>(p, maps, s);
}

template <class T>
cudaError_t local_t(const DeltaParams &p, const DeltaMaps &maps, cudaStream_t s) {
    if constexpr (kPieces<T> == 1)
        if (maps.made) return p.keys <= 64 ? local_k<T, 64, true>(p, maps, s) : local_k<T, 128, true>(p, maps, s);
    return p.keys <= 64 ? local_k<T, 64, false>(p, maps, s) : local_k<T, 128, false>(p, maps, s);
}

}  // namespace

cudaError_t launch_delta_local(dwp_dtype t, const DeltaParams &p, const DeltaMaps &m, cudaStream_t s) {
    if (t == DWP_F32) return local_t<float>(p, m, s);
    return t == DWP_BF16 ? local_t<__nv_bfloat16>(p, m, s) : local_t<__half>(p, m, s);
}

}  // namespace dwp
