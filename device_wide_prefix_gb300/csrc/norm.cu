// Block norm: the root-mean-square norm before and after a block, fused with
// the residual add and its scale (before) and with the gate (after), and its
// gradient.
//
//   v = residual + scale * x            (or x);  sum = v
//   t = v * silu(gate)                  (gate before the norm; else t = v)
//   y = t * rsqrt(mean_group(t^2) + eps) * weight   (* silu(gate) after it)
//
// One block per row and group; a row's elements stay in registers between
// the statistics and the output, so each input is read once and HBM bounds it:
// 8192 x 4096 bf16 with an f32 residual 403 MB in 74 us, 0.80 of the copy rate
// (0.62 with parameters read one by one and loads behind stores).
#include "sequence.cuh"

namespace dwp {

namespace {

// Each of the N values of `v` summed over the block; every thread gets the sums.
// sh: 32 words for each.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float *sh) {
    const int warps = (blockDim.x + 31) / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (warps == 1) return;
    __syncthreads();  // the previous use of sh is over
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) sh[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float s = lane < warps ? sh[k * 32 + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        v[k] = s;
    }
}

template <class T, int V>
__device__ __forceinline__ void load_residual(float (&f)[V], const void *p, int64_t i, bool is_f32) {
    if (is_f32) load_f32<V>(f, static_cast<const float *>(p) + i);
    else load_f32<V>(f, static_cast<const T *>(p) + i);
}
template <class T, int V>
__device__ __forceinline__ void store_residual(void *p, int64_t i, const float (&f)[V], bool is_f32) {
    if (is_f32) store_f32<V>(static_cast<float *>(p) + i, f);
    else store_f32<V>(static_cast<T *>(p) + i, f);
}

template <class T, int V, int K, int kMost, int kBlocks>
__global__ void __launch_bounds__(kMost, kBlocks) norm_kernel(NormParams p) {
    __shared__ float sh[32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x / p.groups;
    const int64_t g0 = int64_t(blockIdx.x % p.groups) * p.group;
    const T *x = static_cast<const T *>(p.x) + row * p.x_row + g0;
    const T *z = p.gate ? static_cast<const T *>(p.gate) + row * p.gate_row + g0 : nullptr;
    T *y = static_cast<T *>(p.y) + row * p.y_row + g0;
    // every load first: a store between them would hold the later ones back
    float v[K][V], gt[K][V], sc[K][V], ss[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t i = (int64_t(k) * blockDim.x + threadIdx.x) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) v[k][j] = 0.0f, gt[k][j] = 1.0f;
        if (i < p.group) {
            load_f32<V>(v[k], x + i);
            if (p.residual) load_residual<T, V>(sc[k], p.residual, row * p.residual_row + g0 + i, p.residual_f32);
            if (z) load_f32<V>(gt[k], z + i);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t i = (int64_t(k) * blockDim.x + threadIdx.x) * V;
        if (i < p.group) {
            if (p.residual) {
                float s[V];
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] = 1.0f;
                if (p.scale) load_params<T, V>(s, p.scale, g0 + i, p.weight_f32);
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] = fmaf(s[j], v[k][j], sc[k][j]);
                store_residual<T, V>(p.sum, row * p.sum_row + g0 + i, v[k], p.residual_f32);
            }
            if (z) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    gt[k][j] = silu(gt[k][j]);
                    if (!p.gate_after) v[k][j] *= gt[k][j];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) ss[0] = fmaf(v[k][j], v[k][j], ss[0]);
    }
    block_sums(ss, sh);
    const float r = rsqrtf(ss[0] / float(p.group) + p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t i = (int64_t(k) * blockDim.x + threadIdx.x) * V;
        if (i < p.group) {
            float o[V], w[V];
            load_params<T, V>(w, p.weight, g0 + i, p.weight_f32);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[j] = v[k][j] * r * w[j];
                if (p.gate_after) o[j] *= gt[k][j];
            }
            store_f32<V>(y + i, o);
        }
    }
}

// Gradient.  With h = t r (r the inverse root mean square) and gw = dy * weight
// (after: dy * silu(gate) * weight):
//   dt = r (gw - h mean(gw h)),  dweight = sum_rows dy h (* silu(gate)).
// Both means come from one reduction (t^2 and gw t).  A block keeps one
// group's columns and walks rows blockIdx.x, + gridDim.x, ..., so the column
// sums stay in registers; each block writes its share and a second kernel
// adds the shares in a fixed order.
//
// A thread holds the raw values of its columns of one row, and loads the next
// row's before it waits for the block's sums.  Wide groups (kWideRow) leave no
// registers for that: there the column sums are in shared memory, each word one
// thread's own, and the weights are read again for each row (8192 x 8192 bf16
// with a gate: 223 us, against 472 with spilled sums).  4096 x 8192 f16 in 8
// groups with a gate: 336 MB in 97 us; issue (0.65 a cycle) and the wait for the
// sums bound it.
template <class T, int V, int K>
struct NormRow {
    Pack<float, V> v32[K];  // the norm's input in f32, or
    Pack<T, V> v[K];        // in the activations' type
    Pack<T, V> dy[K], gate[K];
};

template <class T, int V, int K, bool kWideV, int kMost, int kBlocks, bool kWideRow>
__global__ void __launch_bounds__(kMost, kBlocks) norm_backward_kernel(NormBackwardParams q) {
    __shared__ float sh[64];
    extern __shared__ float sums[];  // kWideRow: [2][threads * K * V], a thread's own words threads apart
    pdl_trigger();
    pdl_wait();
    const NormParams &p = q.n;
    const int64_t g0 = int64_t(blockIdx.y) * p.group;
    const bool gated = p.gate != nullptr;
    constexpr bool kW = kWideRow;
    constexpr int kKept = kW ? 1 : K;
    float dw[kKept][V], ds[kKept][V], w[kKept][V];
    auto slot = [&](int which, int k, int j) -> float & {
        return sums[((which * K + k) * V + j) * int(blockDim.x) + int(threadIdx.x)];
    };
    int at[K];  // this thread's columns; past the group they are read from its start and not used
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = (k * int(blockDim.x) + int(threadIdx.x)) * V;
        in[k] = i < p.group, at[k] = int(g0) + (in[k] ? i : 0);
        if constexpr (kWideRow) {
#pragma unroll
            for (int j = 0; j < V; ++j) slot(0, k, j) = slot(1, k, j) = 0.0f;
        } else {
            load_params<T, V>(w[k], p.weight, at[k], p.weight_f32);
#pragma unroll
            for (int j = 0; j < V; ++j) dw[k][j] = ds[k][j] = 0.0f;
        }
    }
    auto load = [&](NormRow<T, V, K> &r, int64_t row) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (kWideV)
                r.v32[k] = *reinterpret_cast<const Pack<float, V> *>(static_cast<const float *>(q.v) + row * q.v_row + at[k]);
            else r.v[k] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(q.v) + row * q.v_row + at[k]);
            r.dy[k] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(q.grad_out) + row * q.grad_row + at[k]);
            if (gated)
                r.gate[k] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(p.gate) + row * p.gate_row + at[k]);
        }
    };
    NormRow<T, V, K> now, next;
    if (!kWideRow && int64_t(blockIdx.x) < p.rows) load(next, blockIdx.x);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        if constexpr (kWideRow) {
            load(now, row);
        } else {
            now = next;
            load(next, min(row + gridDim.x, p.rows - 1));
        }
        auto vin = [&](int k, int j) { return kWideV ? now.v32[k].e[j] : to_f32<T>(now.v[k].e[j]); };
        float red[2] = {0.0f, 0.0f}, sg[kKept][V];  // sg: sigmoid of the gate
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (kWideRow) load_params<T, V>(w[0], p.weight, at[k], p.weight_f32);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float t = in[k] ? vin(k, j) : 0.0f, gw = to_f32<T>(now.dy[k].e[j]) * w[kWideRow ? 0 : k][j];
                if (gated) {
                    const float zv = to_f32<T>(now.gate[k].e[j]), s = sigmoid(zv);
                    if (!kWideRow) sg[kWideRow ? 0 : k][j] = s;
                    (p.gate_after ? gw : t) *= zv * s;
                }
                red[0] = fmaf(t, t, red[0]);
                red[1] = fmaf(gw, t, red[1]);
            }
        }
        block_sums(red, sh);
        const float r = rsqrtf(red[0] / float(p.group) + p.eps);
        const float m = red[1] * r / float(p.group) * r;  // mean(gw h) r: dt = r gw - t r m
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!in[k]) continue;
            float dz[V], dv[V], add[V], xs[V];
            if constexpr (kW) load_params<T, V>(w[0], p.weight, at[k], p.weight_f32);
            if (q.grad_sum) load_residual<T, V>(add, q.grad_sum, row * q.gsum_row + at[k], q.v_f32);
            if (q.x_in) load_f32<V>(xs, static_cast<const T *>(q.x_in) + row * q.xin_row + at[k]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float v = vin(k, j), zv = gated ? to_f32<T>(now.gate[k].e[j]) : 0.0f;
                const float sig = !gated ? 0.0f : kW ? sigmoid(zv) : sg[kW ? 0 : k][j];
                const float s = gated ? zv * sig : 1.0f, wj = w[kW ? 0 : k][j];
                float g = to_f32<T>(now.dy[k].e[j]), t = v;
                if (gated && !p.gate_after) t *= s;
                const float h = t * r;
                if (gated && p.gate_after) {
                    dz[j] = g * h * wj * silu_slope(zv, sig);
                    g *= s;
                }
                if constexpr (kW) slot(0, k, j) = fmaf(g, h, slot(0, k, j));
                else dw[k][j] = fmaf(g, h, dw[k][j]);
                float d = r * fmaf(-t, m, g * wj);
                if (gated && !p.gate_after) {
                    dz[j] = d * v * silu_slope(zv, sig);
                    d *= s;
                }
                if (q.grad_sum) d += add[j];
                dv[j] = d;
                if (q.x_in) {
                    if constexpr (kW) slot(1, k, j) = fmaf(d, xs[j], slot(1, k, j));
                    else ds[k][j] = fmaf(d, xs[j], ds[k][j]);
                }
            }
            if (gated) store_f32<V>(static_cast<T *>(q.grad_gate) + row * q.ggate_row + at[k], dz);
            if (q.grad_residual) store_residual<T, V>(q.grad_residual, row * q.gres_row + at[k], dv, q.v_f32);
            if (q.grad_x) {
                if (p.scale) {
                    float s[V];
                    load_params<T, V>(s, p.scale, at[k], p.weight_f32);
#pragma unroll
                    for (int j = 0; j < V; ++j) dv[j] *= s[j];
                }
                store_f32<V>(static_cast<T *>(q.grad_x) + row * q.gx_row + at[k], dv);
            }
        }
    }
    float *part = q.partial + int64_t(blockIdx.x) * (q.x_in ? 2 : 1) * p.channels;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!in[k]) continue;
        if constexpr (kWideRow) {
#pragma unroll
            for (int j = 0; j < V; ++j) dw[0][j] = slot(0, k, j), ds[0][j] = slot(1, k, j);
        }
        store_f32<V>(part + at[k], dw[kWideRow ? 0 : k]);
        if (q.x_in) store_f32<V>(part + p.channels + at[k], ds[kWideRow ? 0 : k]);
    }
}

// Threads for a group of `n` elements at V per access and K accesses a thread.
uint32_t threads_for(int64_t n, int v, int k) {
    const int64_t need = (n + int64_t(v) * k - 1) / (int64_t(v) * k);
    return uint32_t((need + 31) / 32 * 32);
}

// The fewest accesses a thread that a block of kMost threads allows.
template <class T, int V, int K, int kMost, int kBlocks>
cudaError_t norm_k(const NormParams &p, cudaStream_t s) {
    return launch_pdl(norm_kernel<T, V, K, kMost, kBlocks>, dim3(uint32_t(p.rows * p.groups)), dim3(threads_for(p.group, V, K)), 0,
                      s, p);
}

template <class T, int V>
cudaError_t norm_v(const NormParams &p, cudaStream_t s) {
    if constexpr (V == 1) {
        if (p.group <= 1024) return norm_k<T, 1, 2, 512, 2>(p, s);
        if (p.group <= 4096) return norm_k<T, 1, 8, 512, 2>(p, s);
        return norm_k<T, 1, 16, 1024, 1>(p, s);
    } else {
        if (p.group <= 512 * V) return norm_k<T, V, 1, 512, 2>(p, s);
        if (p.group <= 1024 * V) return norm_k<T, V, 2, 512, 2>(p, s);
        // 16-bit types have V = 8 and end here; f32 has V = 4
        if constexpr (2048 * V < DWP_NORM_MAX_GROUP)
            if (p.group > 2048 * V) return norm_k<T, V, 32 / V, 512, 1>(p, s);
        return norm_k<T, V, 2, 1024, 1>(p, s);
    }
}

// Shared memory for two sums of the widest group's columns.
constexpr size_t kWideRowBytes = size_t(512) * 32 * 2 * sizeof(float);

// Accesses a thread of the gradient makes for a group of `n` elements, V each.
int64_t backward_accesses(int64_t n, int v) {
    if (v == 1) return n <= 1024 ? 2 : n <= 4096 ? 8 : 32;
    return n <= 512 * v ? 1 : n <= 1024 * v ? 2 : 32 / v;
}

template <class T, int V, bool kWideV>
cudaError_t norm_backward_v(const NormBackwardParams &q, cudaStream_t s) {
    const NormParams &p = q.n;
    const dim3 grid(uint32_t(q.blocks), uint32_t(p.groups));
    const int64_t k = backward_accesses(p.group, V);
    const uint32_t threads = threads_for(p.group, V, int(k));
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(threads), 0, s, q); };
    auto wide = [&](auto kernel) {
        const size_t smem = size_t(threads) * k * V * 2 * sizeof(float);
        if (device_blocks(reinterpret_cast<const void *>(kernel), 512, kWideRowBytes) == 0)
            return cudaErrorInvalidConfiguration;
        return launch_pdl(kernel, grid, dim3(threads), smem, s, q);
    };
    if constexpr (V == 1) {
        if (k == 2) return go(norm_backward_kernel<T, 1, 2, kWideV, 512, 1, false>);
        if (k == 8) return go(norm_backward_kernel<T, 1, 8, kWideV, 512, 1, false>);
        return wide(norm_backward_kernel<T, 1, 32, kWideV, 512, 1, true>);
    } else {
        if (p.group <= 128 * V) return go(norm_backward_kernel<T, V, 1, kWideV, 128, 4, false>);
        if (k == 1) return go(norm_backward_kernel<T, V, 1, kWideV, 512, 1, false>);
        if (k == 2) return wide(norm_backward_kernel<T, V, 2, kWideV, 512, 1, true>);
        return wide(norm_backward_kernel<T, V, 32 / V, kWideV, 512, 1, true>);
    }
}

template <class T, int V>
cudaError_t norm_backward_t(const NormBackwardParams &q, cudaStream_t s) {
    if constexpr (sizeof(T) != 4)
        if (q.v_f32) return norm_backward_v<T, V, true>(q, s);
    return norm_backward_v<T, V, false>(q, s);
}

constexpr int kColThreads = 256;

// out[c] = sum over blocks of part[b][c], c < cols: 32 columns by 8 strands
// of blocks per thread block, the strands joined in order.
__global__ void __launch_bounds__(kColThreads)
    column_sums_kernel(const float *part, int64_t blocks, int64_t cols, ColumnOut o) {
    __shared__ float sh[8][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % 32, strand = threadIdx.x / 32;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t b = strand; b < blocks; b += 8) s += part[b * cols + c];
    }
    sh[strand][lane] = s;
    __syncthreads();
    if (strand == 0 && c < cols) {
        s = sh[0][lane];
#pragma unroll
        for (int k = 1; k < 8; ++k) s += sh[k][lane];
        if (c < o.end[0]) {  // column c is entry c % inner of plane c / inner
            const int64_t inner = o.end[0] / o.planes;
            if (o.out[0]) o.out[0][c % inner * o.planes + c / inner] = s;
        } else if (c < o.end[1]) {
            if (o.out[1]) o.out[1][c - o.end[0]] = s;
        } else if (c < o.end[2]) {
            if (o.out[2]) o.out[2][c - o.end[1]] = s;
        }
    }
}

}  // namespace

cudaError_t launch_column_sums(const float *part, int64_t blocks, int64_t cols, const ColumnOut &o, cudaStream_t s) {
    return launch_pdl(column_sums_kernel, dim3(uint32_t((cols + 31) / 32)), dim3(kColThreads), 0, s, part, blocks,
                      cols, o);
}

int64_t norm_backward_threads(dwp_dtype t, int64_t group, bool vec) {
    const int v = !vec ? 1 : t == DWP_F32 ? 4 : 8;
    return threads_for(group, v, int(backward_accesses(group, v)));
}

cudaError_t launch_norm(dwp_dtype t, const NormParams &p, bool vec, cudaStream_t s) {
    if (t == DWP_F32) return vec ? norm_v<float, 4>(p, s) : norm_v<float, 1>(p, s);
    if (t == DWP_BF16) return vec ? norm_v<__nv_bfloat16, 8>(p, s) : norm_v<__nv_bfloat16, 1>(p, s);
    return vec ? norm_v<__half, 8>(p, s) : norm_v<__half, 1>(p, s);
}

cudaError_t launch_norm_backward(dwp_dtype t, const NormBackwardParams &p, bool vec, cudaStream_t s) {
    if (t == DWP_F32) return vec ? norm_backward_t<float, 4>(p, s) : norm_backward_t<float, 1>(p, s);
    if (t == DWP_BF16) return vec ? norm_backward_t<__nv_bfloat16, 8>(p, s) : norm_backward_t<__nv_bfloat16, 1>(p, s);
    return vec ? norm_backward_t<__half, 8>(p, s) : norm_backward_t<__half, 1>(p, s);
}

}  // namespace dwp
