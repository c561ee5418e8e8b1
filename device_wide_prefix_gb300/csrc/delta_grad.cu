// Gated delta rule, the gradients of a chunk's rows, from the state before it,
// its corrections U, the gradient of the state after it and that of the
// corrections' right sides, dR:
//
//   dA = scale dO U^T (j <= i), decayed;   E = -exp(G_i - G_j) dR_i.U_j (j < i)
//   dQ = scale e^G dO S0^T + dA K
//   Z  = E K - e^G dR S0^T,   Y = e^{G_C - G} U dS1^T + dA^T Q + (beta E)^T K
//   dK = beta Z + Y,   dV = beta dR,   dbeta = dR.V + k.Z
//   dG = q.dQ + beta k.Z - k.Y, and <S1, dS1> at the chunk's last row; dg its
//   sum from the last row down
//
// (dG: G_i is in e^{G_i} q_i and, as e^{G_i} beta_i k_i and e^{-G_i} k_i, in
// what k_i does first and what it does to later rows.)
#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kThreads = 256;

// store(i, j, sum over k < kk of a(i, k) b(k, j)) for i < m, j < n.
template <class FA, class FB, class FS>
__device__ __forceinline__ void delta_product(int m, int n, int kk, FA a, FB b, FS store) {
    const int mt = (m + 3) / 4, nt = (n + 3) / 4;
    for (int e = threadIdx.x; e < mt * nt; e += blockDim.x) {
        const int i0 = e / nt * 4, j0 = e % nt * 4;
        float s[4][4] = {};
        for (int k = 0; k < kk; ++k) {
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = a(min(i0 + i, m - 1), k), y[i] = b(k, min(j0 + i, n - 1));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = fmaf(x[i], y[j], s[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + i < m && j0 + j < n) store(i0 + i, j0 + j, s[i][j]);
    }
}


template <class T>
__global__ void __launch_bounds__(kThreads) delta_grad_kernel(DeltaBackwardParams bp) {
    const DeltaParams &p = bp.f;
    extern __shared__ float sh[];
    __shared__ Sum2 sums[kChunk];
    __shared__ float beta[kChunk], first[kChunk], rest[kChunk], dots[3][kChunk], whole_dot;
    const int keys = p.keys, values = p.values, tid = threadIdx.x;
    float *dw = sh, *cross = dw + kChunk * kChunk, *acc = cross + kChunk * kChunk, *z = acc + kChunk * keys;
    pdl_trigger();
    pdl_wait();
    const int head = blockIdx.y, kh = head / (p.heads / p.key_heads);
    const DeltaChunk c = delta_chunk(p, blockIdx.x);
    if (c.rows == 0) return;
    const int n = c.rows;
    if (tid < 32) {
        delta_sums(sums, [&](int i) { return i < n ? delta_g(p.g, c.batch, c.row + i, head) : 0.0f; });
        __syncwarp();
        for (int i = tid; i < kChunk; i += 32) {
            beta[i] = i < n ? delta_beta<T>(p, c.batch, c.row + i, head) : 0.0f;
            first[i] = expf(sums[i].hi), rest[i] = expf(sum2_less(sums[kChunk - 1], sums[i]));
            dots[0][i] = dots[1][i] = dots[2][i] = 0.0f;
        }
    }
    __syncthreads();
    const int64_t at = int64_t(blockIdx.x) * p.heads + head;
    const int kp = (keys + 7) / 8 * 8;
    const __nv_bfloat16 *P0 = reinterpret_cast<const __nv_bfloat16 *>(p.states + at * kp * values);
    const __nv_bfloat16 *P1 = reinterpret_cast<const __nv_bfloat16 *>(bp.ends + at * kp * values);
    auto S0 = [&](int k, int v) { return __bfloat162float(P0[v * kp + k]) + __bfloat162float(P0[(values + v) * kp + k]); };
    auto S1 = [&](int k, int v) { return __bfloat162float(P1[v * kp + k]) + __bfloat162float(P1[(values + v) * kp + k]); };
    const float *U = p.u + at * kChunk * values, *dR = bp.dr + at * kChunk * values;
    auto q = [&](int i, int k) { return i < n ? to_f32<T>(delta_at<T>(p.q, c.batch, c.row + i, kh)[k]) : 0.0f; };
    auto k_ = [&](int i, int k) { return i < n ? to_f32<T>(delta_at<T>(p.k, c.batch, c.row + i, kh)[k]) : 0.0f; };
    auto go = [&](int i, int j) { return i < n ? to_f32<T>(delta_at<T>(bp.grad_out, c.batch, c.row + i, head)[j]) : 0.0f; };
    delta_product(kChunk, kChunk, values, go, [&](int v, int j) { return U[j * values + v]; }, [&](int i, int j, float s) {
        dw[i * kChunk + j] = j <= i ? p.scale * expf(sum2_less(sums[i], sums[j])) * s : 0.0f;
    });
    delta_product(kChunk, kChunk, values, [&](int i, int v) { return dR[i * values + v]; },
                  [&](int v, int j) { return U[j * values + v]; }, [&](int i, int j, float s) {
                      cross[i * kChunk + j] = j < i ? -expf(sum2_less(sums[i], sums[j])) * s : 0.0f;
                  });
    auto put = [&](const DeltaRows &t, int which, int i, int k, float v) {
        if (p.heads == p.key_heads) delta_at<T>(t, c.batch, c.row + i, head)[k] = from_f32<T>(v);
        else bp.share[((at * 2 + which) * kChunk + i) * keys + k] = v;
    };
    // row i's product with `of`, added to dots[which][i]
    auto dot = [&](int which, auto of) {
        __syncthreads();
        for (int i = tid / 32; i < n; i += kThreads / 32) {
            float s = 0.0f;
            for (int k = tid % 32; k < keys; k += 32) s += of(i, k);
            for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (tid % 32 == 0) dots[which][i] += s;
        }
        __syncthreads();
    };
    // dQ
    delta_product(n, keys, values, go, [&](int v, int k) { return S0(k, v); },
                  [&](int i, int k, float s) { acc[i * keys + k] = p.scale * first[i] * s; });
    __syncthreads();
    delta_product(n, keys, n, [&](int i, int j) { return dw[i * kChunk + j]; }, k_, [&](int i, int k, float s) {
        acc[i * keys + k] += s;
        put(bp.grad_q, 0, i, k, acc[i * keys + k]);
    });
    dot(0, [&](int i, int k) { return q(i, k) * acc[i * keys + k]; });
    // Z
    delta_product(n, keys, values, [&](int i, int v) { return dR[i * values + v]; },
                  [&](int v, int k) { return S0(k, v); },
                  [&](int i, int k, float s) { z[i * keys + k] = -first[i] * s; });
    __syncthreads();
    delta_product(n, keys, n, [&](int i, int j) { return cross[i * kChunk + j]; }, k_,
                  [&](int i, int k, float s) { z[i * keys + k] += s; });
    dot(1, [&](int i, int k) { return k_(i, k) * z[i * keys + k]; });
    // Y, and the part of <S1, dS1> that this chunk wrote
    delta_product(n, keys, values, [&](int i, int v) { return U[i * values + v]; },
                  [&](int v, int k) { return S1(k, v); },
                  [&](int i, int k, float s) { acc[i * keys + k] = rest[i] * s; });
    __syncthreads();
    if (tid < 32) {
        float s = 0.0f;
        for (int i = 0; i < n; ++i)
            for (int k = tid; k < keys; k += 32) s = fmaf(k_(i, k), acc[i * keys + k], s);
        for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid == 0) whole_dot = s;
    }
    __syncthreads();
    if (tid < 32) {
        float s = 0.0f;
        for (int e = tid; e < keys * values; e += 32) s = fmaf(S0(e / values, e % values), S1(e / values, e % values), s);
        for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid == 0) whole_dot = fmaf(first[kChunk - 1], s, whole_dot);
    }
    __syncthreads();
    delta_product(n, keys, n, [&](int j, int i) { return dw[i * kChunk + j]; }, q,
                  [&](int i, int k, float s) { acc[i * keys + k] += s; });
    __syncthreads();
    delta_product(n, keys, n, [&](int j, int i) { return beta[i] * cross[i * kChunk + j]; }, k_,
                  [&](int i, int k, float s) {
                      acc[i * keys + k] += s;
                      put(bp.grad_k, 1, i, k, fmaf(beta[i], z[i * keys + k], acc[i * keys + k]));
                  });
    dot(2, [&](int i, int k) { return k_(i, k) * acc[i * keys + k]; });
    // dV, dbeta, dg
    for (int i = tid / 32; i < n; i += kThreads / 32) {
        float s = 0.0f;
        for (int j = tid % 32; j < values; j += 32) {
            const float d = dR[i * values + j];
            s = fmaf(d, to_f32<T>(delta_at<T>(p.v, c.batch, c.row + i, head)[j]), s);
            delta_at<T>(bp.grad_v, c.batch, c.row + i, head)[j] = from_f32<T>(beta[i] * d);
        }
        for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid % 32 == 0) {
            const float d = s + dots[1][i];
            if (p.beta_f32) *delta_at<float>(bp.grad_beta, c.batch, c.row + i, head) = d;
            else *delta_at<T>(bp.grad_beta, c.batch, c.row + i, head) = from_f32<T>(d);
        }
    }
    if (tid < 32 && bp.grad_g.data) {
        __shared__ Sum2 rev[kChunk];
        delta_sums(rev, [&](int r) {
            const int i = kChunk - 1 - r;
            return i >= n ? 0.0f : dots[0][i] + beta[i] * dots[1][i] - dots[2][i] + (i == n - 1 ? whole_dot : 0.0f);
        });
        __syncwarp();
        for (int i = tid; i < n; i += 32) *delta_at<float>(bp.grad_g, c.batch, c.row + i, head) = rev[kChunk - 1 - i].hi;
    }
}

// grad_q and grad_k of a key head: the sum over its heads' shares, in order.
template <class T>
__global__ void __launch_bounds__(kThreads) delta_share_kernel(DeltaBackwardParams bp) {
    const DeltaParams &p = bp.f;
    pdl_trigger();
    pdl_wait();
    const DeltaChunk c = delta_chunk(p, blockIdx.x);
    const int kh = blockIdx.y, per = p.heads / p.key_heads;
    for (int e = threadIdx.x; e < 2 * c.rows * p.keys; e += kThreads) {
        const int which = e / (c.rows * p.keys), i = e / p.keys % c.rows, k = e % p.keys;
        float s = 0.0f;
        for (int h = 0; h < per; ++h) {
            const int64_t at = int64_t(blockIdx.x) * p.heads + kh * per + h;
            s += bp.share[((at * 2 + which) * kChunk + i) * p.keys + k];
        }
        delta_at<T>(which ? bp.grad_k : bp.grad_q, c.batch, c.row + i, kh)[k] = from_f32<T>(s);
    }
}

constexpr size_t grad_bytes(int keys) { return sizeof(float) * size_t(2 * kChunk * kChunk + 2 * kChunk * keys); }

template <class T>
cudaError_t grad_t(const DeltaBackwardParams &p, cudaStream_t s) {
    const auto kernel = delta_grad_kernel<T>;
    if (device_blocks(reinterpret_cast<const void *>(kernel), kThreads, grad_bytes(128)) == 0)
        return cudaErrorInvalidConfiguration;
    const cudaError_t err = launch_pdl(kernel, dim3(uint32_t(p.f.slots), uint32_t(p.f.heads)), dim3(kThreads),
                                       grad_bytes(p.f.keys), s, p);
    if (err != cudaSuccess || p.f.heads == p.f.key_heads) return err;
    return launch_pdl(delta_share_kernel<T>, dim3(uint32_t(p.f.slots), uint32_t(p.f.key_heads)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_delta_grad(dwp_dtype t, const DeltaBackwardParams &p, cudaStream_t s) {
    if (t == DWP_F32) return grad_t<float>(p, s);
    return t == DWP_BF16 ? grad_t<__nv_bfloat16>(p, s) : grad_t<__half>(p, s);
}

}  // namespace dwp
