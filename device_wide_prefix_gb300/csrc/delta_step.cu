// Gated delta rule, the single-token form: each row of a batch moves its
// sequence's state on by one step and reads it out.  The state is read and
// written once, which is nearly all of the traffic.
//
//   p = S^T k, r = S^T q;  u = beta (v - a p);  o = scale (a r + (q.k) u);  S = a S + k u^T
//
// so the state stays in registers between one reduction and its update.  64 rows
// x 32 heads of 128 x 128 (268 MB of states) take 57 us, 0.70 of the copy rate;
// 256 rows 216 us, 0.73.  Blocks of 128 threads and 32 columns: 256 threads took
// 66 and 244 us, 16 columns 56 and 281, 64 columns 63 and 240.
#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kThreads = 128;
constexpr int kLanes = 8;                   // neighbouring accesses of a state's row
constexpr int kGroups = kThreads / kLanes;  // state rows at once
constexpr int kRows = 128 / kGroups;        // state rows a thread

template <class T, int V>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(DeltaStepParams p) {
    __shared__ alignas(16) float part[kThreads / 32][2][kLanes * V];
    __shared__ float dots[kThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int head = blockIdx.y, kh = head / (p.heads / p.key_heads), tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int lane = tid % kLanes, group = tid / kLanes, j0 = (int(blockIdx.z) * kLanes + lane) * V;
    const int64_t slot = p.slots ? p.slots[row] : row;
    T *out = delta_at<T>(p.out, 0, row, head);
    if (slot < 0 || slot >= p.num_slots) {
        if (group == 0 && j0 < p.values) {
            const float zero[V] = {};
            store_f32<V>(out + j0, zero);
        }
        return;
    }
    float *state = p.state + slot * p.state_slot + int64_t(head) * p.keys * p.values + j0;
    const T *q = delta_at<T>(p.q, 0, row, kh), *k = delta_at<T>(p.k, 0, row, kh);
    float S[kRows][V], kk[kRows], qq[kRows];
    const bool in = j0 < p.values;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int i = r * kGroups + group;
        kk[r] = qq[r] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) S[r][v] = 0.0f;
        if (i < p.keys) {
            kk[r] = to_f32<T>(k[i]), qq[r] = to_f32<T>(q[i]);
            if (in) load_f32<V>(S[r], state + int64_t(i) * p.values);
        }
    }
    const float a = expf(delta_g(p.g, 0, row, head));
    const float beta = p.beta_f32 ? *delta_at<float>(p.beta, 0, row, head) : to_f32<T>(*delta_at<T>(p.beta, 0, row, head));
    float v[V] = {};
    if (in) load_f32<V>(v, delta_at<T>(p.v, 0, row, head) + j0);
    float sk[V] = {}, sq[V] = {}, qk = 0.0f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        qk = fmaf(qq[r], kk[r], qk);
#pragma unroll
        for (int j = 0; j < V; ++j) sk[j] = fmaf(S[r][j], kk[r], sk[j]), sq[j] = fmaf(S[r][j], qq[r], sq[j]);
    }
#pragma unroll
    for (int o = kLanes; o < 32; o *= 2) {
        qk += __shfl_xor_sync(0xffffffffu, qk, o);
#pragma unroll
        for (int j = 0; j < V; ++j)
            sk[j] += __shfl_xor_sync(0xffffffffu, sk[j], o), sq[j] += __shfl_xor_sync(0xffffffffu, sq[j], o);
    }
    const int warp = tid / 32;
    if (tid % 32 < kLanes) {
        store_f32<V>(&part[warp][0][lane * V], sk);
        store_f32<V>(&part[warp][1][lane * V], sq);
        dots[warp] = qk;
    }
    __syncthreads();
    qk = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) sk[j] = sq[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        float a_k[V], a_q[V];
        load_f32<V>(a_k, &part[w][0][lane * V]);
        load_f32<V>(a_q, &part[w][1][lane * V]);
        qk += dots[w];
#pragma unroll
        for (int j = 0; j < V; ++j) sk[j] += a_k[j], sq[j] += a_q[j];
    }
    if (!in) return;
    float u[V], o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) u[j] = beta * (v[j] - a * sk[j]), o[j] = p.scale * fmaf(qk, u[j], a * sq[j]);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int i = r * kGroups + group;
        if (i < p.keys) {
            float s[V];
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = fmaf(kk[r], u[j], a * S[r][j]);
            store_f32<V>(state + int64_t(i) * p.values, s);
        }
    }
    if (group == 0) store_f32<V>(out + j0, o);
}

template <class T, int V>
cudaError_t step_v(const DeltaStepParams &p, cudaStream_t s) {
    const uint32_t blocks = uint32_t((p.values + kLanes * V - 1) / (kLanes * V));
    return launch_pdl(delta_step_kernel<T, V>, dim3(uint32_t(p.batch), uint32_t(p.heads), blocks), dim3(kThreads), 0, s, p);
}

template <class T>
cudaError_t step_t(const DeltaStepParams &p, cudaStream_t s) {
    return p.wide ? step_v<T, 4>(p, s) : step_v<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_delta_step(dwp_dtype t, const DeltaStepParams &p, cudaStream_t s) {
    if (t == DWP_F32) return step_t<float>(p, s);
    return t == DWP_BF16 ? step_t<__nv_bfloat16>(p, s) : step_t<__half>(p, s);
}

}  // namespace dwp
