// Layer norm over each of `groups` equal parts of a row, fused with the
// residual add before it, and its gradient.
//
//   v = residual + x (or x);  sum = v
//   h = (v - mean) r,  r = 1 / sqrt(mean((v - mean)^2) + eps),  y = h weight + bias
//
// A team of threads holds one row's group in registers, so each input is read
// once: up to a warp's threads where the group fits them, a block above.  Mean
// and squares come from one reduction: each thread has the mean and the sum of
// squares about it of its own values, and two such pairs join as
//   d = mean_b - mean_a,  M2 = M2_a + M2_b + d^2 n_a n_b / n,
// which loses nothing where the mean is far from zero.
#include "sequence.cuh"

namespace dwp {

namespace {

// Count, mean, squares about the mean; and for the gradient the mean of a
// second value and the products of both about their means.
template <bool kTwo>
struct Moments {
    float n, mean, m2, mean_g, c;
};

template <bool kTwo>
__device__ __forceinline__ Moments<kTwo> join(const Moments<kTwo> &a, const Moments<kTwo> &b) {
    Moments<kTwo> r;
    r.n = a.n + b.n;
    const float share = r.n > 0.0f ? __fdividef(b.n, r.n) : 0.0f, d = b.mean - a.mean, w = a.n * share;
    r.mean = fmaf(d, share, a.mean);
    r.m2 = fmaf(d * d, w, a.m2 + b.m2);
    if constexpr (kTwo) {
        const float e = b.mean_g - a.mean_g;
        r.mean_g = fmaf(e, share, a.mean_g);
        r.c = fmaf(d * e, w, a.c + b.c);
    }
    return r;
}

template <bool kTwo>
__device__ __forceinline__ Moments<kTwo> shuffled(const Moments<kTwo> &a, int o) {
    Moments<kTwo> r;
    r.n = __shfl_xor_sync(0xffffffffu, a.n, o);
    r.mean = __shfl_xor_sync(0xffffffffu, a.mean, o);
    r.m2 = __shfl_xor_sync(0xffffffffu, a.m2, o);
    if constexpr (kTwo) {
        r.mean_g = __shfl_xor_sync(0xffffffffu, a.mean_g, o);
        r.c = __shfl_xor_sync(0xffffffffu, a.c, o);
    }
    return r;
}

// The team's moments, in every thread of it.  sh: two sets of 32, used in turn.
template <bool kTwo, bool kBlock>
__device__ __forceinline__ Moments<kTwo> team_moments(Moments<kTwo> m, int team, Moments<kTwo> *sh, int turn) {
    if constexpr (!kBlock) {
        for (int o = team / 2; o > 0; o /= 2) m = join(m, shuffled(m, o));
        return m;
    } else {
#pragma unroll
        for (int o = 16; o > 0; o /= 2) m = join(m, shuffled(m, o));
        const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
        Moments<kTwo> *set = sh + turn % 2 * 32;  // the other set may still be read
        if (lane == 0) set[threadIdx.x / 32] = m;
        __syncthreads();
        m = lane < warps ? set[lane] : Moments<kTwo>{};
#pragma unroll
        for (int o = 16; o > 0; o /= 2) m = join(m, shuffled(m, o));
        return m;
    }
}

template <class T, int V>
__device__ __forceinline__ void load_either(float (&f)[V], const void *p, int64_t i, bool is_f32) {
    if (is_f32) load_f32<V>(f, static_cast<const float *>(p) + i);
    else load_f32<V>(f, static_cast<const T *>(p) + i);
}
template <class T, int V>
__device__ __forceinline__ void store_either(void *p, int64_t i, const float (&f)[V], bool is_f32) {
    if (is_f32) store_f32<V>(static_cast<float *>(p) + i, f);
    else store_f32<V>(static_cast<T *>(p) + i, f);
}

// A thread's own moments of K accesses of V values, `in` telling which count.
template <int V, int K, bool kTwo>
__device__ __forceinline__ Moments<kTwo> own_moments(const float (&v)[K][V], const float (*g)[V], const bool (&in)[K]) {
    Moments<kTwo> m = {};
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (in[k]) {
            m.n += float(V);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                m.mean += v[k][j];
                if constexpr (kTwo) m.mean_g += g[k][j];
            }
        }
    const float inv = m.n > 0.0f ? __fdividef(1.0f, m.n) : 0.0f;
    m.mean *= inv;
    if constexpr (kTwo) m.mean_g *= inv;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (in[k]) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = v[k][j] - m.mean;
                m.m2 = fmaf(d, d, m.m2);
                if constexpr (kTwo) m.c = fmaf(d, g[k][j] - m.mean_g, m.c);
            }
        }
    return m;
}

template <class T, int V, int K, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) layer_norm_kernel(LayerNormParams p) {
    __shared__ Moments<false> sh[kBlock ? 64 : 1];
    pdl_trigger();
    pdl_wait();
    const int team = kBlock ? int(blockDim.x) : p.team;
    const int64_t which = kBlock ? int64_t(blockIdx.x) : (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / team;
    const int t = kBlock ? int(threadIdx.x) : int(threadIdx.x) % team;
    const int64_t row = which / p.groups;
    const bool live = kBlock || row < p.rows;
    const int64_t g0 = which % p.groups * p.group;
    float v[K][V], more[K][V];
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t i = (int64_t(k) * team + t) * V;
        in[k] = live && i < p.group;
        if (in[k]) {
            load_f32<V>(v[k], static_cast<const T *>(p.x) + row * p.x_row + g0 + i);
            if (p.residual) load_either<T, V>(more[k], p.residual, row * p.residual_row + g0 + i, p.residual_f32);
        }
    }
    if (p.residual)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (in[k]) {
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] += more[k][j];
                store_either<T, V>(p.sum, row * p.sum_row + g0 + (int64_t(k) * team + t) * V, v[k], p.residual_f32);
            }
    const Moments<false> m = team_moments<false, kBlock>(own_moments<V, K, false>(v, nullptr, in), team, sh, 0);
    const float r = rsqrtf(m.m2 / float(p.group) + p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (in[k]) {
            const int64_t i = g0 + (int64_t(k) * team + t) * V;
            float o[V], w[V], b[V];
            if (p.weight) load_params<T, V>(w, p.weight, i, p.weight_f32);
            if (p.bias) load_params<T, V>(b, p.bias, i, p.weight_f32);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[j] = (v[k][j] - m.mean) * r;
                if (p.weight) o[j] *= w[j];
                if (p.bias) o[j] += b[j];
            }
            store_f32<V>(static_cast<T *>(p.y) + row * p.y_row + i, o);
        }
}

// Gradient, with gw = dy weight:
//   dv = r (gw - mean(gw) - h mean(gw h)),  dweight = sum_rows dy h,  dbias = sum_rows dy
// The products of gw and v about their means come with the same reduction.  A
// block keeps one group's columns and its teams walk the rows, so the column
// sums stay with the thread; the teams of a block add theirs in order, each
// block writes its share, and a second kernel adds the shares in order.
template <class T, int V, int K, bool kBlock, bool kWideV>
__global__ void __launch_bounds__(kBlock ? 512 : 256) layer_norm_backward_kernel(LayerNormBackwardParams q) {
    __shared__ Moments<true> sh[kBlock ? 64 : 1];
    extern __shared__ float sums[];  // K > 1: [2][K * V][threads]; else the teams' sums at the end
    pdl_trigger();
    pdl_wait();
    const LayerNormParams &p = q.n;
    constexpr bool kShared = K > 1;  // column sums in shared memory, each word one thread's own
    using TV = typename std::conditional<kWideV, float, T>::type;
    const int threads = blockDim.x, tid = threadIdx.x, team = kBlock ? threads : p.team, t = tid % team;
    const int teams = threads / team;
    const int64_t g0 = int64_t(blockIdx.y) * p.group;
    float dw[kShared ? 1 : V], db[kShared ? 1 : V];
    auto slot = [&](int which, int k, int j) -> float & { return sums[((which * K + k) * V + j) * threads + tid]; };
    int at[K];
    bool own[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = (k * team + t) * V;
        own[k] = i < p.group, at[k] = int(g0) + (own[k] ? i : 0);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (kShared) slot(0, k, j) = slot(1, k, j) = 0.0f;
            else dw[j] = db[j] = 0.0f;
        }
    }
    const int64_t stride = int64_t(gridDim.x) * teams;
    int turn = 0;
    // whole blocks go round together: the moments' shuffles take every lane
    for (int64_t r0 = int64_t(blockIdx.x) * teams; r0 < p.rows; r0 += stride, ++turn) {
        const int64_t row = r0 + tid / team;
        const bool live = row < p.rows;
        float v[K][V], dy[K][V], gw[K][V];
        bool in[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            in[k] = own[k] && live;
            if (in[k]) {
                load_f32<V>(v[k], static_cast<const TV *>(q.v) + row * q.v_row + at[k]);
                load_f32<V>(dy[k], static_cast<const T *>(q.grad_out) + row * q.grad_row + at[k]);
                if (p.weight) load_params<T, V>(gw[k], p.weight, at[k], p.weight_f32);
#pragma unroll
                for (int j = 0; j < V; ++j) gw[k][j] = p.weight ? gw[k][j] * dy[k][j] : dy[k][j];
            }
        }
        const Moments<true> m = team_moments<true, kBlock>(own_moments<V, K, true>(v, gw, in), team, sh, turn);
        const float inv = 1.0f / float(p.group), r = rsqrtf(m.m2 * inv + p.eps), c = m.c * inv * r * r;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!in[k]) continue;
            float add[V];
            if (q.grad_sum) load_f32<V>(add, static_cast<const TV *>(q.grad_sum) + row * q.gsum_row + at[k]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = v[k][j] - m.mean;
                if constexpr (kShared) {
                    slot(0, k, j) = fmaf(dy[k][j] * d, r, slot(0, k, j));
                    slot(1, k, j) += dy[k][j];
                } else {
                    dw[j] = fmaf(dy[k][j] * d, r, dw[j]);
                    db[j] += dy[k][j];
                }
                gw[k][j] = r * (gw[k][j] - m.mean_g - d * c);
                if (q.grad_sum) gw[k][j] += add[j];
            }
            if (q.grad_residual)
                store_f32<V>(static_cast<TV *>(q.grad_residual) + row * q.gres_row + at[k], gw[k]);
            if (q.grad_x) store_f32<V>(static_cast<T *>(q.grad_x) + row * q.gx_row + at[k], gw[k]);
        }
    }
    if (!q.partial) return;
    if constexpr (!kShared) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) slot(0, 0, j) = dw[j], slot(1, 0, j) = db[j];
    }
    __syncthreads();
    if (tid >= team) return;
    float *part = q.partial + int64_t(blockIdx.x) * 2 * p.channels;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!own[k]) continue;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float s[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[j] = 0.0f;
                for (int o = 0; o < teams; ++o) s[j] += sums[((which * K + k) * V + j) * threads + o * team + t];
            }
            store_f32<V>(part + which * p.channels + at[k], s);
        }
    }
}

// How a group is spread: accesses a thread, and threads of a team.
struct Spread {
    int k, team;
    bool block;
};
Spread spread(int64_t group, int v, int most_threads) {
    const int64_t pieces = (group + v - 1) / v;
    if (pieces <= 32) {
        int team = 1;
        while (team < pieces) team *= 2;
        return {1, team, false};
    }
    if (pieces <= 64) return {2, 32, false};
    for (int k : {1, 2, 4, 8, 16}) {
        const int64_t threads = (pieces + k - 1) / k;
        if (threads <= most_threads) return {k, int((threads + 31) / 32 * 32), true};
    }
    return {32, most_threads, true};
}

constexpr int kTeamThreads = 256;
constexpr size_t kSumBytes = size_t(2) * 16384 * sizeof(float);

template <class T, int V, int K, bool kBlock>
cudaError_t forward_k(const LayerNormParams &p, cudaStream_t s) {
    const int64_t work = p.rows * p.groups;
    if (kBlock) return launch_pdl(layer_norm_kernel<T, V, K, true>, dim3(uint32_t(work)), dim3(p.team), 0, s, p);
    const int64_t teams = kTeamThreads / p.team;
    return launch_pdl(layer_norm_kernel<T, V, K, false>, dim3(uint32_t((work + teams - 1) / teams)), dim3(kTeamThreads), 0,
                      s, p);
}

template <class T, int V>
cudaError_t forward_v(LayerNormParams p, cudaStream_t s) {
    const Spread a = spread(p.group, V, 1024);
    p.team = a.team;
    if (!a.block) return a.k == 1 ? forward_k<T, V, 1, false>(p, s) : forward_k<T, V, 2, false>(p, s);
    switch (a.k) {
        case 1: return forward_k<T, V, 1, true>(p, s);
        case 2: return forward_k<T, V, 2, true>(p, s);
        case 4: return forward_k<T, V, 4, true>(p, s);
        default: return forward_k<T, V, 16, true>(p, s);
    }
}

template <class T, int V, int K, bool kBlock, bool kWideV>
cudaError_t backward_k(const LayerNormBackwardParams &q, cudaStream_t s) {
    const auto kernel = layer_norm_backward_kernel<T, V, K, kBlock, kWideV>;
    const int threads = kBlock ? q.n.team : kTeamThreads;
    const size_t smem = size_t(2) * K * V * threads * sizeof(float);
    if (smem > 48u * 1024 && device_blocks(reinterpret_cast<const void *>(kernel), 512, kSumBytes) == 0)
        return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, dim3(uint32_t(q.blocks), uint32_t(q.n.groups)), dim3(threads), smem, s, q);
}

template <class T, int V, bool kWideV>
cudaError_t backward_v(LayerNormBackwardParams q, cudaStream_t s) {
    const Spread a = spread(q.n.group, V, 512);
    q.n.team = a.team;
    if (!a.block) return a.k == 1 ? backward_k<T, V, 1, false, kWideV>(q, s) : backward_k<T, V, 2, false, kWideV>(q, s);
    switch (a.k) {
        case 1: return backward_k<T, V, 1, true, kWideV>(q, s);
        case 2: return backward_k<T, V, 2, true, kWideV>(q, s);
        case 4: return backward_k<T, V, 4, true, kWideV>(q, s);
        case 8: return backward_k<T, V, 8, true, kWideV>(q, s);
        default: return backward_k<T, V, 32, true, kWideV>(q, s);
    }
}

template <class T, int V>
cudaError_t backward_t(const LayerNormBackwardParams &q, cudaStream_t s) {
    if constexpr (sizeof(T) != 4)
        if (q.v_f32) return backward_v<T, V, true>(q, s);
    return backward_v<T, V, false>(q, s);
}

}  // namespace

int64_t layer_norm_teams(dwp_dtype t, int64_t group, bool vec) {
    const Spread a = spread(group, !vec ? 1 : t == DWP_F32 ? 4 : 8, 512);
    return a.block ? 1 : kTeamThreads / a.team;
}

cudaError_t launch_layer_norm(dwp_dtype t, const LayerNormParams &p, bool vec, cudaStream_t s) {
    if (t == DWP_F32) return vec ? forward_v<float, 4>(p, s) : forward_v<float, 1>(p, s);
    if (t == DWP_BF16) return vec ? forward_v<__nv_bfloat16, 8>(p, s) : forward_v<__nv_bfloat16, 1>(p, s);
    return vec ? forward_v<__half, 8>(p, s) : forward_v<__half, 1>(p, s);
}

cudaError_t launch_layer_norm_backward(dwp_dtype t, const LayerNormBackwardParams &p, bool vec, cudaStream_t s) {
    if (t == DWP_F32) return vec ? backward_t<float, 4>(p, s) : backward_t<float, 1>(p, s);
    if (t == DWP_BF16) return vec ? backward_t<__nv_bfloat16, 8>(p, s) : backward_t<__nv_bfloat16, 1>(p, s);
    return vec ? backward_t<__half, 8>(p, s) : backward_t<__half, 1>(p, s);
}

}  // namespace dwp
