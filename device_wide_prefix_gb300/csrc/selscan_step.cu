// Selective state space scan, the single-token form: each row of a batch
// moves its sequence's state on by one step and reads it out.  The state is
// read and written once, and that is nearly all of the traffic: at batch 256 x
// 4096 channels x 16 states 142 MB in 26 us, 0.81 of the copy rate.  Two batch
// rows a thread, 32 warps an SM; four states a lane instead of eight took 36
// us (twice the softplus and addresses), four rows 30, one row 27.
#include "selscan.cuh"

namespace dwp {

namespace {

constexpr int kStepThreads = 128;
constexpr int kStepRows = 2;  // batch rows a thread takes: their loads are all in flight together

// Place of a lane's state j within its channel.
template <int NL>
__device__ __forceinline__ int state_at(int nl, int j) {
    return (j / 4 * NL + nl) * 4 + j % 4;
}

// A lane's 4 P values from x; zeros past `states`.
template <class E, int NL, int P, bool kWide>
__device__ __forceinline__ void load_pieces(float (&v)[4 * P], const E *x, int nl, int states) {
    if constexpr (kWide) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float f[4];
            load_f32<4, E>(f, x + state_at<NL>(nl, 4 * i));
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = f[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4 * P; ++j) {
            const int n = state_at<NL>(nl, j);
            v[j] = n < states ? to_f32<E>(x[n]) : 0.0f;
        }
    }
}

// NL neighbouring lanes share a channel.  A lane has P pieces of four states,
// NL pieces apart, so that each access of the lanes of a channel is one run of
// memory; more states a lane spread the work per channel (softplus, addresses)
// over more of them.  kWide: a piece is one aligned access in A, B, C and the
// states, and they fill all pieces.
template <class T, int NL, int P, bool kWide>
__global__ void __launch_bounds__(kStepThreads, 8) scan_step_kernel(ScanStepParams p) {
    constexpr int kCh = kStepThreads / NL;
    pdl_trigger();
    pdl_wait();
    const int nl = threadIdx.x % NL;
    constexpr int kN = 4 * P;  // states of a lane
    const uint32_t g = blockIdx.y / p.group_blocks;
    const int64_t cg = int64_t(blockIdx.y % p.group_blocks) * kCh + threadIdx.x / NL;
    const bool own = cg < p.group;
    const int64_t c = int64_t(g) * p.group + (own ? cg : p.group - 1);
    const int64_t b0 = int64_t(blockIdx.x) * kStepRows;

    float A[kN], h[kStepRows][kN], B[kStepRows][kN], C[kStepRows][kN], d[kStepRows], u[kStepRows], z[kStepRows];
    int64_t slot[kStepRows];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int64_t b = min(b0 + i, p.batch - 1);
        slot[i] = p.slots ? p.slots[b] : b;
    }
    load_pieces<float, NL, P, kWide>(A, p.A + c * p.states, nl, p.states);
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int64_t b = min(b0 + i, p.batch - 1);
        // a padding row keeps nothing, and A stands for its state in the loads:
        // any slot may be another row's to write
        if (slot[i] < 0 || slot[i] >= p.num_slots) slot[i] = -1;
        const float *from = slot[i] < 0 ? p.A : p.state + slot[i] * p.state_slot;
        load_pieces<float, NL, P, kWide>(h[i], from + c * p.states, nl, p.states);
        load_pieces<T, NL, P, kWide>(B[i], static_cast<const T *>(p.B) + b * p.b_row + g * p.b_group, nl, p.states);
        load_pieces<T, NL, P, kWide>(C[i], static_cast<const T *>(p.C) + b * p.c_row + g * p.c_group, nl, p.states);
        d[i] = to_f32<T>(static_cast<const T *>(p.dt)[b * p.dt_row + c]);
        u[i] = to_f32<T>(static_cast<const T *>(p.u)[b * p.u_row + c]);
        z[i] = p.z ? to_f32<T>(static_cast<const T *>(p.z)[b * p.z_row + c]) : 0.0f;
    }
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, D = p.D ? p.D[c] : 0.0f;
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        float delta = d[i] + bias;
        if (p.softplus) delta = softplus_poly(delta);
        // delta, not A, times log2(e): 0 times any finite A is then 0
        const float x = delta * u[i], rate = delta * kLog2e;
        float y = 0.0f;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            h[i][j] = fmaf(ex2(rate * A[j]), h[i][j], x * B[i][j]);
            y = fmaf(C[i][j], h[i][j], y);
        }
#pragma unroll
        for (int o = NL / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (!own || b0 + i >= p.batch) continue;
        if (slot[i] >= 0) {
            float *to = p.state + slot[i] * p.state_slot + c * p.states;
            if constexpr (kWide) {
#pragma unroll
                for (int k = 0; k < P; ++k)
                    store_f32<4>(to + state_at<NL>(nl, 4 * k), {h[i][4 * k], h[i][4 * k + 1], h[i][4 * k + 2], h[i][4 * k + 3]});
            } else {
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    if (state_at<NL>(nl, j) < p.states) to[state_at<NL>(nl, j)] = h[i][j];
            }
        }
        if (nl == 0) {
            y = fmaf(D, u[i], y);
            if (p.z) y *= silu(z[i]);
            static_cast<T *>(p.out)[(b0 + i) * p.out_row + c] = from_f32<T>(slot[i] < 0 ? 0.0f : y);
        }
    }
}

template <class T, int NL, int P>
cudaError_t step_nl(ScanStepParams p, cudaStream_t s) {
    constexpr int kCh = kStepThreads / NL;
    p.group_blocks = uint32_t((p.group + kCh - 1) / kCh);
    const dim3 grid(uint32_t((p.batch + kStepRows - 1) / kStepRows), uint32_t(p.groups * p.group_blocks));
    if (p.wide && p.states == 4 * NL * P)
        return launch_pdl(scan_step_kernel<T, NL, P, true>, grid, dim3(kStepThreads), 0, s, p);
    return launch_pdl(scan_step_kernel<T, NL, P, false>, grid, dim3(kStepThreads), 0, s, p);
}

template <class T>
cudaError_t step_t(const ScanStepParams &p, cudaStream_t s) {
    if (p.states <= 8) return step_nl<T, 2, 1>(p, s);
    if (p.states <= 16) return step_nl<T, 2, 2>(p, s);
    if (p.states <= 32) return step_nl<T, 4, 2>(p, s);
    if (p.states <= 64) return step_nl<T, 8, 2>(p, s);
    return step_nl<T, 16, 2>(p, s);
}

}  // namespace

cudaError_t launch_selscan_step(dwp_dtype t, const ScanStepParams &p, cudaStream_t s) {
    if (t == DWP_F32) return step_t<float>(p, s);
    if (t == DWP_BF16) return step_t<__nv_bfloat16>(p, s);
    return step_t<__half>(p, s);
}

}  // namespace dwp
