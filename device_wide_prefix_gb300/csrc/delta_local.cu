// Gated delta rule, what a chunk needs of itself alone: the inverse
// T = (1 + L)^-1, L the strictly lower part of diag(beta) M, and the weights A,
// each in two planes of bf16.
//
// One product of [K; Q] with K gives k_i.k_j in the lanes of the first 64 rows
// and q_i.k_j in the others, for all heads that share the keys; teams of 128
// threads take the heads in turn.  A thread has one row; the rows of L go to
// shared memory.  The inverse is that of its two diagonal blocks of 32, by
// substitution with a thread a column, and -T22 L21 T11 below them: a third of
// the steps that all 64 columns at once would wait for one after another.
#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kTeam = 128;
constexpr int kHalf = kChunk / 2;
constexpr int kPitch = kChunk + 4;  // words a row of L and T: rows start on 16 bytes, in other banks

template <class T, int KD, int kTeams>
constexpr size_t local_bytes = 1024 + size_t(kPieces<T>) * 2 * kChunk * KD * 2 + size_t(kTeams) * kChunk * kPitch * 4;

template <class T, int KD, bool kWide, int kTeams>
__global__ void __launch_bounds__(kTeam * kTeams, 4 / kTeams) delta_local_kernel(DeltaParams p) {
    extern __shared__ char raw[];
    __shared__ Sum2 sums_[kTeams][kChunk];
    __shared__ float beta_[kTeams][kChunk];
    __shared__ uint64_t bar;
    __shared__ uint32_t tmem;
    constexpr uint32_t kLo = 2 * kChunk * KD * 2;
    char *tile = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
    pdl_trigger();
    pdl_wait();
    const DeltaChunk c = delta_chunk(p, blockIdx.x);
    if (c.rows == 0) return;
    const int lane = threadIdx.x % 32, warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);
    const int team = warp / 4, tid = threadIdx.x % kTeam;
    const int kh = blockIdx.y, per = p.heads / p.key_heads;
    float *L = reinterpret_cast<float *>(tile + kPieces<T> * kLo) + team * kChunk * kPitch;  // and T, block by block
    Sum2 *sums = sums_[team];
    float *beta = beta_[team];
    auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(kTeam) : "memory"); };
    // a head's log decays, and betas, by the team's first and last warp
    float g[2], b[2];
    auto load_rows = [&](int h) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = lane + 32 * i;
            const bool in = r < c.rows && h < per;
            if (warp % 4 == 0) g[i] = in ? delta_g(p.g, c.batch, c.row + r, kh * per + h) : 0.0f;
            if (warp % 4 == 3) b[i] = in ? delta_beta<T>(p, c.batch, c.row + r, kh * per + h) : 0.0f;
        }
    };
    load_tile<T, kWide, 2 * kChunk, KD, kTeam * kTeams>(threadIdx.x, tile, kLo, 0, p.k, c.batch, c.row, kh, c.rows, p.keys);
    load_tile<T, kWide, 2 * kChunk, KD, kTeam * kTeams>(threadIdx.x, tile, kLo, kChunk, p.q, c.batch, c.row, kh, c.rows, p.keys);
    load_rows(team);
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem, kChunk);
    copies_done();
    fence_proxy_async_smem();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t d = tmem;
    if (warp == 0 && elect_one()) {
        const Operand<2 * kChunk, false> hi(tile), lo(tile + kLo);
        product_ss<kChunk, KD>(d, hi, hi, false);
        if constexpr (kPieces<T> == 2) {
            product_ss<kChunk, KD>(d, hi, lo, true);
            product_ss<kChunk, KD>(d, lo, hi, true);
        }
        mma_commit(&bar);
    }
    bool ok = true;
    const int row = tid % kChunk;  // of the chunk, as key or as query
    for (int h = team; h < per; h += kTeams) {
        const int64_t at = int64_t(blockIdx.x) * p.heads + kh * per + h;
        char *T_out = reinterpret_cast<char *>(p.inverse + at * kChunk * kChunk);
        char *A_out = reinterpret_cast<char *>(p.weights + at * kChunk * kChunk);
        sync();
        if (warp % 4 == 0) {
            Sum2 s[2];
            delta_sums(s, g);
            sums[lane] = s[0], sums[lane + 32] = s[1];
        }
        if (warp % 4 == 3) beta[lane] = b[0], beta[lane + 32] = b[1];
        load_rows(h + kTeams);
        sync();
        if (h == team) {
            ok = mma_wait(&bar, 0);
            tmem_fence_after();
        }
        const Sum2 mine = sums[row];
        const float scale = ok ? tid < kChunk ? beta[row] : 1.0f : __int_as_float(0x7fffffff);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t v[32];
            tmem_load<32>(v, d + (uint32_t(warp % 4) << 21) + half * 32);
            tmem_ready();
#pragma unroll
            for (int j0 = 0; j0 < 32; j0 += 8) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int col = half * 32 + j0 + j;
                    const bool in = tid < kChunk ? col < row : col <= row;
                    f[j] = in ? scale * __expf(sum2_less(mine, sums[col])) * __uint_as_float(v[j0 + j]) : 0.0f;
                }
                if (tid < kChunk) {
                    float4 *to = reinterpret_cast<float4 *>(L + row * kPitch + half * 32 + j0);
                    to[0] = make_float4(f[0], f[1], f[2], f[3]);
                    to[1] = make_float4(f[4], f[5], f[6], f[7]);
                } else {
                    store_pieces(A_out, p.u || kPieces<T> == 2 ? A_out + kChunk * kTileRow : nullptr,
                                 tile_piece(uint32_t(row), uint32_t(half * 4 + j0 / 8)), f);
                }
            }
        }
        sync();
        // the diagonal blocks' inverses: column `lane` of block `warp`, kept in registers, then in the block's place
        if (warp % 4 < 2) {
            float *B = L + warp % 4 * kHalf * (kPitch + 1);
            float x[kHalf];
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                float s0 = i == lane ? 1.0f : 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(B + i * kPitch + j);
                    s0 = fmaf(-l.x, x[j], s0);
                    if (j + 1 < i) s1 = fmaf(-l.y, x[j + 1], s1);
                    if (j + 2 < i) s2 = fmaf(-l.z, x[j + 2], s2);
                    if (j + 3 < i) s3 = fmaf(-l.w, x[j + 3], s3);
                }
                x[i] = (s0 + s1) + (s2 + s3);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kHalf; ++i) B[i * kPitch + lane] = x[i];
        }
        sync();
        // below them: first L21 T11 (into the unused upper right), then -T22 of it in L21's place
        const int r = tid / 4, c0 = tid % 4 * 8;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            const float *a = L + (kHalf + r) * kPitch + (pass ? kHalf : 0), *from = L + (pass ? kHalf : 0) + c0;
            float s[8] = {};
#pragma unroll
            for (int k = 0; k < kHalf; k += 4) {
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
            float4 *to = reinterpret_cast<float4 *>(L + (pass ? kHalf + r : r) * kPitch + (pass ? 0 : kHalf) + c0);
            to[0] = pass ? make_float4(-s[0], -s[1], -s[2], -s[3]) : make_float4(s[0], s[1], s[2], s[3]);
            to[1] = pass ? make_float4(-s[4], -s[5], -s[6], -s[7]) : make_float4(s[4], s[5], s[6], s[7]);
            sync();
        }
#pragma unroll
        for (int e = tid; e < kChunk * kChunk / 8; e += kTeam) {
            const int i = e / 8, j0 = e % 8 * 8;
            float f[8];
            load_f32<8>(f, L + i * kPitch + j0);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = i < kHalf && j0 >= kHalf ? 0.0f : f[j];
            store_pieces(T_out, T_out + kChunk * kTileRow, tile_piece(uint32_t(i), uint32_t(j0 / 8)), f);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 0) tmem_free(d, kChunk);
}

template <class T, int KD, bool kWide, int kTeams>
cudaError_t local_n(const DeltaParams &p, cudaStream_t s) {
    const auto kernel = delta_local_kernel<T, KD, kWide, kTeams>;
    constexpr size_t bytes = local_bytes<T, KD, kTeams>;
    if (device_blocks(reinterpret_cast<const void *>(kernel), kTeam * kTeams, bytes) == 0) return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, dim3(uint32_t(p.slots), uint32_t(p.key_heads)), dim3(kTeam * kTeams), bytes, s, p);
}

template <class T, int KD, bool kWide>
cudaError_t local_k(const DeltaParams &p, cudaStream_t s) {
    return p.heads == p.key_heads ? local_n<T, KD, kWide, 1>(p, s) : local_n<T, KD, kWide, 2>(p, s);
}

template <class T>
cudaError_t local_t(const DeltaParams &p, cudaStream_t s) {
    if (p.keys <= 64) return p.wide ? local_k<T, 64, true>(p, s) : local_k<T, 64, false>(p, s);
    return p.wide ? local_k<T, 128, true>(p, s) : local_k<T, 128, false>(p, s);
}

}  // namespace

cudaError_t launch_delta_local(dwp_dtype t, const DeltaParams &p, cudaStream_t s) {
    if (t == DWP_F32) return local_t<float>(p, s);
    return t == DWP_BF16 ? local_t<__nv_bfloat16>(p, s) : local_t<__half>(p, s);
}

}  // namespace dwp
