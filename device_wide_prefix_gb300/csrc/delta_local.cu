// Gated delta rule, what a chunk needs of itself alone: the inverse
// T = (1 + strictly lower part of diag(beta) M)^-1 and the weights A.
#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kThreads = 256;

template <class T>
__global__ void __launch_bounds__(kThreads) delta_local_kernel(DeltaParams p) {
    extern __shared__ float sh[];
    __shared__ Sum2 sums[kChunk];
    __shared__ float beta[kChunk];
    float *tk = sh, *tq = tk + kChunk * p.keys, *sys = tq + kChunk * p.keys, *inv = sys + kChunk * (kChunk + 1);
    pdl_trigger();
    pdl_wait();
    const int head = blockIdx.y, kh = head / (p.heads / p.key_heads);
    const DeltaChunk c = delta_chunk(p, blockIdx.x);
    if (c.rows == 0) return;
    const int tid = threadIdx.x;
    if (tid < 32) delta_sums(sums, [&](int i) { return i < c.rows ? delta_g(p.g, c.batch, c.row + i, head) : 0.0f; });
    if (tid >= 64 && tid < 128) beta[tid - 64] = tid - 64 < c.rows ? delta_beta<T>(p, c.batch, c.row + tid - 64, head) : 0.0f;
    for (int e = tid; e < kChunk * p.keys; e += kThreads) {
        const int i = e / p.keys, j = e % p.keys;
        tk[e] = i < c.rows ? to_f32<T>(delta_at<T>(p.k, c.batch, c.row + i, kh)[j]) : 0.0f;
        tq[e] = i < c.rows ? to_f32<T>(delta_at<T>(p.q, c.batch, c.row + i, kh)[j]) : 0.0f;
    }
    __syncthreads();
    const int64_t at = (int64_t(blockIdx.x) * p.heads + head) * kChunk * kChunk;
    const int keys = p.keys;
    delta_product(kChunk, kChunk, keys, [&](int i, int k) { return tk[i * keys + k]; },
                  [&](int k, int j) { return tk[j * keys + k]; }, [&](int i, int j, float s) {
                      sys[i * (kChunk + 1) + j] = j < i ? beta[i] * expf(sum2_less(sums[i], sums[j])) * s : 0.0f;
                  });
    delta_product(kChunk, kChunk, keys, [&](int i, int k) { return tq[i * keys + k]; },
                  [&](int k, int j) { return tk[j * keys + k]; }, [&](int i, int j, float s) {
                      p.weights[at + i * kChunk + j] = j <= i ? expf(sum2_less(sums[i], sums[j])) * s : 0.0f;
                  });
    __syncthreads();
    // column tid of the inverse, from the top down
    if (tid < kChunk)
        for (int i = 0; i < kChunk; ++i) {
            float s = i == tid ? 1.0f : 0.0f;
            for (int j = tid; j < i; ++j) s = fmaf(-sys[i * (kChunk + 1) + j], inv[j * kChunk + tid], s);
            inv[i * kChunk + tid] = s;
        }
    __syncthreads();
    for (int e = tid; e < kChunk * kChunk; e += kThreads) p.inverse[at + e] = inv[e];
}

template <class T>
cudaError_t local_t(const DeltaParams &p, cudaStream_t s) {
    const size_t smem = sizeof(float) * (2 * kChunk * p.keys + kChunk * (kChunk + 1) + kChunk * kChunk);
    if (device_blocks(reinterpret_cast<const void *>(delta_local_kernel<T>), kThreads,
                      sizeof(float) * (2 * kChunk * 128 + kChunk * (kChunk + 1) + kChunk * kChunk)) == 0)
        return cudaErrorInvalidConfiguration;
    return launch_pdl(delta_local_kernel<T>, dim3(uint32_t(p.slots), uint32_t(p.heads)), dim3(kThreads), smem, s, p);
}

}  // namespace

cudaError_t launch_delta_local(dwp_dtype t, const DeltaParams &p, cudaStream_t s) {
    if (t == DWP_F32) return local_t<float>(p, s);
    return t == DWP_BF16 ? local_t<__nv_bfloat16>(p, s) : local_t<__half>(p, s);
}

}  // namespace dwp
