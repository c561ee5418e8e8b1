// Gated delta rule, the states from chunk to chunk, and their gradients back.
#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kThreads = 256;
constexpr int kCols = 32;  // values of a block: the columns of a state do not meet

constexpr size_t chain_bytes(int keys) {
    return sizeof(float) * size_t(keys * kCols + 2 * kChunk * kCols + kChunk * keys);
}

template <class T, bool kBack>
__global__ void __launch_bounds__(kThreads) delta_chain_kernel(DeltaBackwardParams bp) {
    const DeltaParams &p = bp.f;
    extern __shared__ float sh[];
    __shared__ Sum2 sums[kChunk];
    __shared__ float beta[kChunk], first[kChunk], rest[kChunk];
    const int keys = p.keys, v0 = blockIdx.z * kCols, cols = min(kCols, p.values - v0), tid = threadIdx.x;
    float *S = sh, *R = S + keys * kCols, *U = R + kChunk * kCols, *tk = U + kChunk * kCols;
    pdl_trigger();
    pdl_wait();
    const int head = blockIdx.y, kh = head / (p.heads / p.key_heads);
    const int64_t seq = blockIdx.x;
    int64_t batch, row0, rows, slot0;
    delta_sequence(p, seq, batch, row0, rows, slot0);
    const int64_t state_at = (seq * p.heads + head) * keys * p.values + v0;
    const float *from = kBack ? bp.grad_final : p.initial;
    float *to = kBack ? bp.grad_initial : p.final;
    for (int e = tid; e < keys * cols; e += kThreads) {
        const int k = e / cols, j = e % cols;
        S[k * kCols + j] = from ? from[state_at + int64_t(k) * p.values + j] : 0.0f;
    }
    const int64_t chunks = (rows + kChunk - 1) / kChunk;
    for (int64_t cc = 0; cc < chunks; ++cc) {
        const int64_t c = kBack ? chunks - 1 - cc : cc, row = row0 + c * kChunk;
        const int n = int(min(rows - c * kChunk, int64_t(kChunk)));
        const int64_t at = (slot0 + c) * p.heads + head;
        __syncthreads();
        if (tid < 32) {
            delta_sums(sums, [&](int i) { return i < n ? delta_g(p.g, batch, row + i, head) : 0.0f; });
            __syncwarp();
            for (int i = tid; i < kChunk; i += 32) {
                beta[i] = i < n ? delta_beta<T>(p, batch, row + i, head) : 0.0f;
                first[i] = expf(sums[i].hi), rest[i] = expf(sum2_less(sums[kChunk - 1], sums[i]));
            }
        }
        for (int e = tid; e < kChunk * keys; e += kThreads)
            tk[e] = e / keys < n ? to_f32<T>(delta_at<T>(p.k, batch, row + e / keys, kh)[e % keys]) : 0.0f;
        if (kBack ? bp.ends != nullptr : p.states != nullptr)
            for (int e = tid; e < keys * cols; e += kThreads)
                (kBack ? bp.ends : p.states)[at * keys * p.values + int64_t(e / cols) * p.values + v0 + e % cols] =
                    S[e / cols * kCols + e % cols];
        __syncthreads();
        const float whole = first[kChunk - 1];
        const float *inv = p.inverse + at * kChunk * kChunk, *weights = p.weights + at * kChunk * kChunk;
        auto value = [&](const DeltaRows &t, int i, int j) {
            return i < n ? to_f32<T>(delta_at<T>(t, batch, row + i, head)[v0 + j]) : 0.0f;
        };
        auto query = [&](int i, int k) { return i < n ? to_f32<T>(delta_at<T>(p.q, batch, row + i, kh)[k]) : 0.0f; };
        if constexpr (!kBack) {
            delta_product(kChunk, cols, keys, [&](int i, int k) { return tk[i * keys + k]; },
                          [&](int k, int j) { return S[k * kCols + j]; }, [&](int i, int j, float s) {
                              R[i * kCols + j] = i < n ? beta[i] * (value(p.v, i, j) - first[i] * s) : 0.0f;
                          });
            __syncthreads();
            delta_product(kChunk, cols, kChunk, [&](int i, int k) { return inv[i * kChunk + k]; },
                          [&](int k, int j) { return R[k * kCols + j]; }, [&](int i, int j, float s) {
                              U[i * kCols + j] = s;
                              if (p.u) p.u[at * kChunk * p.values + i * p.values + v0 + j] = s;
                          });
            __syncthreads();
            delta_product(n, cols, keys, query, [&](int k, int j) { return S[k * kCols + j]; },
                          [&](int i, int j, float s) { R[i * kCols + j] = first[i] * s; });
            __syncthreads();
            delta_product(n, cols, kChunk, [&](int i, int k) { return weights[i * kChunk + k]; },
                          [&](int k, int j) { return U[k * kCols + j]; }, [&](int i, int j, float s) {
                              delta_at<T>(p.out, batch, row + i, head)[v0 + j] = from_f32<T>(p.scale * (R[i * kCols + j] + s));
                          });
            __syncthreads();
            delta_product(keys, cols, kChunk, [&](int k, int i) { return tk[i * keys + k]; },
                          [&](int i, int j) { return rest[i] * U[i * kCols + j]; },
                          [&](int k, int j, float s) { S[k * kCols + j] = fmaf(whole, S[k * kCols + j], s); });
        } else {
            delta_product(kChunk, cols, keys, [&](int i, int k) { return tk[i * keys + k]; },
                          [&](int k, int j) { return S[k * kCols + j]; },
                          [&](int i, int j, float s) { R[i * kCols + j] = i < n ? rest[i] * s : 0.0f; });
            __syncthreads();
            delta_product(kChunk, cols, kChunk, [&](int i, int k) { return weights[k * kChunk + i]; },
                          [&](int k, int j) { return value(bp.grad_out, k, j); },
                          [&](int i, int j, float s) { R[i * kCols + j] += p.scale * s; });
            __syncthreads();
            delta_product(kChunk, cols, kChunk, [&](int i, int k) { return inv[k * kChunk + i]; },
                          [&](int k, int j) { return R[k * kCols + j]; }, [&](int i, int j, float s) {
                              U[i * kCols + j] = s;
                              bp.dr[at * kChunk * p.values + i * p.values + v0 + j] = s;
                          });
            __syncthreads();
            delta_product(keys, cols, kChunk, [&](int k, int i) { return first[i] * beta[i] * tk[i * keys + k]; },
                          [&](int i, int j) { return U[i * kCols + j]; },
                          [&](int k, int j, float s) { S[k * kCols + j] = fmaf(whole, S[k * kCols + j], -s); });
            __syncthreads();
            delta_product(keys, cols, n, [&](int k, int i) { return query(i, k); },
                          [&](int i, int j) { return p.scale * first[i] * value(bp.grad_out, i, j); },
                          [&](int k, int j, float s) { S[k * kCols + j] += s; });
        }
    }
    __syncthreads();
    if (to)
        for (int e = tid; e < keys * cols; e += kThreads)
            to[state_at + int64_t(e / cols) * p.values + e % cols] = S[e / cols * kCols + e % cols];
}

template <class T, bool kBack>
cudaError_t chain_t(const DeltaBackwardParams &p, cudaStream_t s) {
    const auto kernel = delta_chain_kernel<T, kBack>;
    if (device_blocks(reinterpret_cast<const void *>(kernel), kThreads, chain_bytes(128)) == 0)
        return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, dim3(uint32_t(p.f.sequences), uint32_t(p.f.heads), uint32_t((p.f.values + kCols - 1) / kCols)),
                      dim3(kThreads), chain_bytes(p.f.keys), s, p);
}

template <bool kBack>
cudaError_t chain(dwp_dtype t, const DeltaBackwardParams &p, cudaStream_t s) {
    if (t == DWP_F32) return chain_t<float, kBack>(p, s);
    return t == DWP_BF16 ? chain_t<__nv_bfloat16, kBack>(p, s) : chain_t<__half, kBack>(p, s);
}

}  // namespace

cudaError_t launch_delta_chain(dwp_dtype t, const DeltaParams &p, cudaStream_t s) {
    DeltaBackwardParams b = {};
    b.f = p;
    return chain<false>(t, b, s);
}
cudaError_t launch_delta_chain_back(dwp_dtype t, const DeltaBackwardParams &p, cudaStream_t s) {
    return chain<true>(t, p, s);
}

}  // namespace dwp
