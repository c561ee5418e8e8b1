// Gated delta rule, what a chunk needs of itself alone: the inverse
// T = (1 + L)^-1, L the strictly lower part of diag(beta) M, and the weights A,
// each in two planes of bf16.
//
// One product of [K; Q] with K gives k_i.k_j in the lanes of the first 64 rows
// and q_i.k_j in the others, for all heads that share the keys.  A thread has
// one row; the rows of L go to shared memory.  The inverse is that of its two
// diagonal blocks of 32, by substitution with a thread a column, and
// -T22 L21 T11 below them: a third of the steps that all 64 columns at once
// would wait for one after another.
#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kThreads = 128;
constexpr int kHalf = kChunk / 2;
constexpr int kPitch = kChunk + 4;  // words a row of L and T: rows start on 16 bytes, in other banks

template <class T, int KD>
constexpr size_t local_bytes = 1024 + size_t(kPieces<T>) * 2 * kChunk * KD * 2 + size_t(2) * kChunk * kPitch * 4;

template <class T, int KD, bool kWide>
__global__ void __launch_bounds__(kThreads) delta_local_kernel(DeltaParams p) {
    extern __shared__ char raw[];
    __shared__ Sum2 sums[kChunk];
    __shared__ float beta[kChunk];
    __shared__ uint64_t bar;
    __shared__ uint32_t tmem;
    constexpr uint32_t kLo = 2 * kChunk * KD * 2;
    char *tile = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
    float *L = reinterpret_cast<float *>(tile + kPieces<T> * kLo), *inv = L + kChunk * kPitch;
    pdl_trigger();
    pdl_wait();
    const DeltaChunk c = delta_chunk(p, blockIdx.x);
    if (c.rows == 0) return;
    const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
    const int kh = blockIdx.y, per = p.heads / p.key_heads;
    load_tile<T, kWide, 2 * kChunk, KD, kThreads>(tile, kLo, 0, p.k, c.batch, c.row, kh, c.rows, p.keys);
    load_tile<T, kWide, 2 * kChunk, KD, kThreads>(tile, kLo, kChunk, p.q, c.batch, c.row, kh, c.rows, p.keys);
    if (tid == 0) {
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
    const bool ok = mma_wait(&bar, 0);
    tmem_fence_after();
    const int row = tid % kChunk;  // of the chunk, as key or as query
    for (int h = 0; h < per; ++h) {
        const int head = kh * per + h;
        const int64_t at = int64_t(blockIdx.x) * p.heads + head;
        __nv_bfloat16 *T_out = reinterpret_cast<__nv_bfloat16 *>(p.inverse + at * kChunk * kChunk);
        __nv_bfloat16 *A_out = reinterpret_cast<__nv_bfloat16 *>(p.weights + at * kChunk * kChunk);
        __syncthreads();
        if (warp == 0)
            delta_sums(sums, [&](int i) { return i < c.rows ? delta_g(p.g, c.batch, c.row + i, head) : 0.0f; });
        if (tid >= kChunk) {
            const int i = tid - kChunk;
            beta[i] = i < c.rows ? delta_beta<T>(p, c.batch, c.row + i, head) : 0.0f;
        }
        __syncthreads();
        const Sum2 mine = sums[row];
        const float scale = ok ? tid < kChunk ? beta[row] : 1.0f : __int_as_float(0x7fffffff);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t v[32];
            tmem_load<32>(v, d + (uint32_t(warp) << 21) + half * 32);
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
                    char *to = reinterpret_cast<char *>(A_out + row * kChunk + half * 32 + j0);
                    store_pieces(to, p.u || kPieces<T> == 2 ? to + kChunk * kChunk * 2 : nullptr, 0, f);
                }
            }
        }
        __syncthreads();
        // the diagonal blocks' inverses: column `lane` of block `warp`, kept in registers
        if (warp < 2) {
            const float *B = L + warp * kHalf * (kPitch + 1);
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
                inv[(warp * kHalf + i) * kPitch + warp * kHalf + lane] = x[i];
            }
        }
        __syncthreads();
        // below them: first L21 T11 (into the unused upper right), then -T22 of it
        const int r = tid / 4, c0 = tid % 4 * 8;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            const float *a = pass ? inv + (kHalf + r) * kPitch + kHalf : L + (kHalf + r) * kPitch;
            const float *b = pass ? inv + kHalf : inv;
            float s[8] = {};
#pragma unroll 8
            for (int k = 0; k < kHalf; ++k) {
                const float x = a[k];
                const float4 y0 = *reinterpret_cast<const float4 *>(b + k * kPitch + c0);
                const float4 y1 = *reinterpret_cast<const float4 *>(b + k * kPitch + c0 + 4);
                s[0] = fmaf(x, y0.x, s[0]), s[1] = fmaf(x, y0.y, s[1]), s[2] = fmaf(x, y0.z, s[2]), s[3] = fmaf(x, y0.w, s[3]);
                s[4] = fmaf(x, y1.x, s[4]), s[5] = fmaf(x, y1.y, s[5]), s[6] = fmaf(x, y1.z, s[6]), s[7] = fmaf(x, y1.w, s[7]);
            }
            float *to = pass ? inv + (kHalf + r) * kPitch + c0 : inv + r * kPitch + kHalf + c0;
#pragma unroll
            for (int j = 0; j < 8; ++j) to[j] = pass ? -s[j] : s[j];
            __syncthreads();
        }
        for (int e = tid; e < kChunk * kChunk / 8; e += kThreads) {
            const int i = e / 8, j0 = e % 8 * 8;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = i < kHalf && j0 >= kHalf ? 0.0f : inv[i * kPitch + j0 + j];
            char *to = reinterpret_cast<char *>(T_out + i * kChunk + j0);
            store_pieces(to, to + kChunk * kChunk * 2, 0, f);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 0) tmem_free(d, kChunk);
}

template <class T, int KD, bool kWide>
cudaError_t local_k(const DeltaParams &p, cudaStream_t s) {
    const auto kernel = delta_local_kernel<T, KD, kWide>;
    if (device_blocks(reinterpret_cast<const void *>(kernel), kThreads, local_bytes<T, KD>) == 0)
        return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, dim3(uint32_t(p.slots), uint32_t(p.key_heads)), dim3(kThreads), local_bytes<T, KD>, s, p);
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
