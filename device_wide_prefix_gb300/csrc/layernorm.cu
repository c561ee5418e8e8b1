// Layer norm over each of `groups` equal parts of a row, fused with the
// residual add before it, and its gradient.
//
//   v = residual + x (or x);  sum = v
//   h = (v - mean) r,  r = 1 / sqrt(mean((v - mean)^2) + eps),  y = h weight + bias
//
// A team of threads holds one row's group in registers, so each input is read
// once: up to a warp's threads where the group fits them, a block above.  Sums
// are taken about means: a warp finds its mean, then its squares about it, and
// warps join by
//   M2 = sum M2_w + n_w (mean_w - mean)^2,
// so a mean far from zero costs nothing, and a block meets once a row.
//
// With a residual memory bounds the forward: 8192 x 4096 bf16 onto an f32 one (403
// MB) takes 77 us, 0.77 of the copy rate; 8 rows 2 us, the rest of a call is the
// host's.  Without one a block's load, its warps' meeting and its store are too
// little to hide one another: 53 us where the bytes take 20, 8192 wide 149 of 40,
// 16384 wide 237 of 79.
// The gradient of the same (537 MB) 124 us, 0.64: it holds a row's values, its
// gradients and the columns' sums, and waits for each row's moments.  4099 x 32
// groups of 128 in f16 36 us, 0.41: few warps a row's loads are spread over.
#include "sequence.cuh"

namespace dwp {

namespace {

// Mean and squares about it; and for the gradient the mean of a second value
// and the products of both about their means.
template <bool kTwo>
struct Moments {
    float mean, m2, mean_g, c;
};

template <int N>
__device__ __forceinline__ void team_sums(float (&v)[N], int team) {
    for (int o = team / 2; o > 0; o /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// Elements of a group of n that a warp of a block has, K accesses of V a thread.
template <int V, int K>
__device__ __forceinline__ float warp_count(int64_t n, int warp) {
    int64_t s = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t left = n - (int64_t(k) * blockDim.x + warp * 32) * V;
        s += left < 0 ? 0 : left > 32 * V ? 32 * V : left;
    }
    return float(int(s));
}

// The team's moments of K accesses of V values, `in` telling which count, in
// every thread.  n: the group's elements, mine: this warp's.  sh: two sets of
// 32, used in turn.
template <int V, int K, bool kTwo, bool kBlock>
__device__ __forceinline__ Moments<kTwo> team_moments(const float (&v)[K][V], const float (*g)[V], const bool (&in)[K], int team,
                                                      float n, float mine, Moments<kTwo> *sh, int turn) {
    constexpr int N = kTwo ? 2 : 1;
    float s[N] = {};
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (in[k])
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[0] += v[k][j];
                if constexpr (kTwo) s[1] += g[k][j];
            }
    team_sums(s, kBlock ? 32 : team);
    const float inv = mine > 0.0f ? __fdividef(1.0f, mine) : 0.0f;
    Moments<kTwo> m = {};
    m.mean = s[0] * inv;
    if constexpr (kTwo) m.mean_g = s[1] * inv;
    float q[N] = {};
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (in[k])
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = v[k][j] - m.mean;
                q[0] = fmaf(d, d, q[0]);
                if constexpr (kTwo) q[1] = fmaf(d, g[k][j] - m.mean_g, q[1]);
            }
    team_sums(q, kBlock ? 32 : team);
    m.m2 = q[0];
    if constexpr (kTwo) m.c = q[1];
    if constexpr (kBlock) {
        const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
        if (warps == 1) return m;
        Moments<kTwo> *set = sh + turn % 2 * 32;  // the other set may still be read
        if (lane == 0) set[threadIdx.x / 32] = m;
        __syncthreads();
        const Moments<kTwo> w = lane < warps ? set[lane] : Moments<kTwo>{};
        const float count = lane < warps ? warp_count<V, K>(int64_t(n), lane) : 0.0f;
        const float all = __fdividef(1.0f, n);
        s[0] = w.mean * count;
        if constexpr (kTwo) s[1] = w.mean_g * count;
        team_sums(s, 32);
        m.mean = s[0] * all;
        if constexpr (kTwo) m.mean_g = s[1] * all;
        const float d = (w.mean - m.mean) * count;
        q[0] = fmaf(d, w.mean - m.mean, w.m2);
        if constexpr (kTwo) q[1] = fmaf(d, w.mean_g - m.mean_g, w.c);
        team_sums(q, 32);
        m.m2 = q[0];
        if constexpr (kTwo) m.c = q[1];
    }
    return m;
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

template <class T, int V, int K, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 1024 : 256, kBlock ? 1 : 4) layer_norm_kernel(LayerNormParams p) {
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
    const float n = float(int(p.group)), mine = kBlock ? warp_count<V, K>(p.group, threadIdx.x / 32) : n;
    const Moments<false> m = team_moments<V, K, false, kBlock>(v, nullptr, in, team, n, mine, sh, 0);
    const float r = rsqrtf(m.m2 / n + p.eps);
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
// sums stay with the thread (of 4 accesses a thread and more: in shared memory);
// the teams of a block add theirs in order, each block writes its share, and a
// second kernel adds the shares in order.  A second block on the SM hides a
// row's loads better than the next row read ahead does, whose registers spill:
// 8192 x 4096 bf16 with an f32 residual 128 us against 155 (three blocks: 186).
template <class T, class TV, int V, int K>
struct LayerNormRow {
    Pack<TV, V> v[K];
    Pack<T, V> dy[K];
};

template <class T, int V, int K, int kMost, bool kBlock, bool kWideV>
__global__ void __launch_bounds__(kMost, kBlock ? 512 / kMost : K == 1 ? 4 : 2) layer_norm_backward_kernel(LayerNormBackwardParams q) {
    __shared__ Moments<true> sh[kBlock ? 64 : 1];
    extern __shared__ float sums[];  // kShared: [2][K * V][threads]; else the teams' sums at the end
    pdl_trigger();
    pdl_wait();
    const LayerNormParams &p = q.n;
    constexpr bool kShared = K > 2;  // column sums in shared memory, each word one thread's own
    using TV = typename std::conditional<kWideV, float, T>::type;
    const int threads = blockDim.x, tid = threadIdx.x, team = kBlock ? threads : p.team, t = tid % team;
    const int teams = threads / team;
    const int64_t g0 = int64_t(blockIdx.y) * p.group;
    const float n = float(int(p.group)), mine = kBlock ? warp_count<V, K>(p.group, tid / 32) : n;
    float dw[kShared ? 1 : K][V], db[kShared ? 1 : K][V];
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
            else dw[k][j] = db[k][j] = 0.0f;
        }
    }
    auto load = [&](LayerNormRow<T, TV, V, K> &r, int64_t row) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            r.v[k] = *reinterpret_cast<const Pack<TV, V> *>(static_cast<const TV *>(q.v) + row * q.v_row + at[k]);
            r.dy[k] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(q.grad_out) + row * q.grad_row + at[k]);
        }
    };
    const int64_t stride = int64_t(gridDim.x) * teams;
    int turn = 0;
    LayerNormRow<T, TV, V, K> now;
    // whole blocks go round together: the moments' shuffles take every lane
    for (int64_t r0 = int64_t(blockIdx.x) * teams; r0 < p.rows; r0 += stride, ++turn) {
        const int64_t row = r0 + tid / team;
        const bool live = row < p.rows;
        load(now, min(row, p.rows - 1));
        Pack<TV, V> add[K];
        if (q.grad_sum)
#pragma unroll
            for (int k = 0; k < K; ++k)
                add[k] = *reinterpret_cast<const Pack<TV, V> *>(static_cast<const TV *>(q.grad_sum) +
                                                                min(row, p.rows - 1) * q.gsum_row + at[k]);
        float v[K][V], gw[K][V];
        bool in[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            in[k] = own[k] && live;
            float w[V];
            if (p.weight) load_params<T, V>(w, p.weight, at[k], p.weight_f32);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[k][j] = to_f32<TV>(now.v[k].e[j]);
                gw[k][j] = p.weight ? w[j] * to_f32<T>(now.dy[k].e[j]) : to_f32<T>(now.dy[k].e[j]);
            }
        }
        const Moments<true> m = team_moments<V, K, true, kBlock>(v, gw, in, team, n, mine, sh, turn);
        const float inv = __fdividef(1.0f, n), r = rsqrtf(m.m2 * inv + p.eps), c = m.c * inv * r * r;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!in[k]) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = v[k][j] - m.mean, dy = to_f32<T>(now.dy[k].e[j]);
                if constexpr (kShared) {
                    slot(0, k, j) = fmaf(dy * d, r, slot(0, k, j));
                    slot(1, k, j) += dy;
                } else {
                    dw[k][j] = fmaf(dy * d, r, dw[k][j]);
                    db[k][j] += dy;
                }
                gw[k][j] = r * (gw[k][j] - m.mean_g - d * c);
                if (q.grad_sum) gw[k][j] += to_f32<TV>(add[k].e[j]);
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
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) slot(0, k, j) = dw[k][j], slot(1, k, j) = db[k][j];
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

// How a group is spread: accesses a thread, and threads of a team (a block, or
// up to a warp of it).
struct Spread {
    int k, team;
    bool block;
};
Spread few(int64_t pieces) {
    int team = 1;
    while (team < pieces && team < 32) team *= 2;
    return {pieces <= 32 ? 1 : 2, team, false};
}
Spread spread(int64_t group, int v) {
    const int64_t pieces = (group + v - 1) / v;
    if (pieces <= 64) return few(pieces);
    for (int k : {1, 2, 4, 16}) {
        const int64_t threads = (pieces + k - 1) / k;
        if (threads <= 1024) return {k, int((threads + 31) / 32 * 32), true};
    }
    return {16, 1024, true};
}
// The gradient has more to hold: 256 threads up to 4 accesses each, so that two
// blocks share an SM, and 512 above.
Spread spread_backward(int64_t group, int v) {
    const int64_t pieces = (group + v - 1) / v;
    if (pieces <= 64) return few(pieces);
    int k = pieces <= 256 ? 1 : pieces <= 512 ? 2 : pieces <= 2048 ? 4 : pieces <= 4096 ? 8 : 32;
    return {k, int(((pieces + k - 1) / k + 31) / 32 * 32), true};
}

constexpr int kTeamThreads = 256;
constexpr size_t kSumBytes = size_t(2) * 16384 * sizeof(float);

template <class T, int V, int K, bool kBlock>
cudaError_t forward_k(const LayerNormParams &p, cudaStream_t s) {
    const int64_t work = p.rows * p.groups;
    const auto kernel = layer_norm_kernel<T, V, K, kBlock>;
    if constexpr (kBlock) return launch_pdl(kernel, dim3(uint32_t(work)), dim3(p.team), 0, s, p);
    const int64_t teams = kTeamThreads / p.team;
    return launch_pdl(kernel, dim3(uint32_t((work + teams - 1) / teams)), dim3(kTeamThreads), 0, s, p);
}

template <class T, int V>
cudaError_t forward_v(LayerNormParams p, cudaStream_t s) {
    const Spread a = spread(p.group, V);
    p.team = a.team;
    if (!a.block) return a.k == 1 ? forward_k<T, V, 1, false>(p, s) : forward_k<T, V, 2, false>(p, s);
    if (a.k == 1) return forward_k<T, V, 1, true>(p, s);
    if (a.k == 2) return forward_k<T, V, 2, true>(p, s);
    // groups of at most 16384: 8 an access end here, 4 an access below
    if constexpr (V <= 4)
        if (a.k == 4) return forward_k<T, V, 4, true>(p, s);
    if constexpr (V == 1) return forward_k<T, V, 16, true>(p, s);
    return cudaErrorInvalidConfiguration;
}

template <class T, int V, int K, int kMost, bool kBlock, bool kWideV>
cudaError_t backward_k(const LayerNormBackwardParams &q, cudaStream_t s) {
    const auto kernel = layer_norm_backward_kernel<T, V, K, kMost, kBlock, kWideV>;
    const int threads = kBlock ? q.n.team : kTeamThreads;
    const size_t smem = size_t(2) * K * V * threads * sizeof(float);
    if (smem > 48u * 1024 && device_blocks(reinterpret_cast<const void *>(kernel), kMost, kSumBytes) == 0)
        return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, dim3(uint32_t(q.blocks), uint32_t(q.n.groups)), dim3(threads), smem, s, q);
}

template <class T, int V, bool kWideV>
cudaError_t backward_v(LayerNormBackwardParams q, cudaStream_t s) {
    const Spread a = spread_backward(q.n.group, V);
    q.n.team = a.team;
    if (!a.block) return a.k == 1 ? backward_k<T, V, 1, 256, false, kWideV>(q, s) : backward_k<T, V, 2, 256, false, kWideV>(q, s);
    if (a.k == 1) return backward_k<T, V, 1, 256, true, kWideV>(q, s);
    if (a.k == 2) return backward_k<T, V, 2, 256, true, kWideV>(q, s);
    if (a.k == 4) return a.team <= 256 ? backward_k<T, V, 4, 256, true, kWideV>(q, s) : backward_k<T, V, 4, 512, true, kWideV>(q, s);
    // groups of at most 16384: 16-bit types, 8 an access, end here
    if constexpr (V <= 4)
        if (a.k == 8) return backward_k<T, V, 8, 512, true, kWideV>(q, s);
    if constexpr (V == 1) return backward_k<T, V, 32, 512, true, kWideV>(q, s);
    return cudaErrorInvalidConfiguration;
}

template <class T, int V>
cudaError_t backward_t(const LayerNormBackwardParams &q, cudaStream_t s) {
    if constexpr (sizeof(T) != 4)
        if (q.v_f32) return backward_v<T, V, true>(q, s);
    return backward_v<T, V, false>(q, s);
}

}  // namespace

int64_t layer_norm_teams(dwp_dtype t, int64_t group, bool vec, int64_t &per_sm) {
    const Spread a = spread_backward(group, !vec ? 1 : t == DWP_F32 ? 4 : 8);
    per_sm = !a.block && a.k == 1 ? 4 : a.team <= 256 ? 2 : 1;
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
