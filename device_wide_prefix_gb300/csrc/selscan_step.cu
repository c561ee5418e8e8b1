// Selective state space scan, the single-token form: each row of a batch
// moves its sequence's state on by one step and reads it out.  The state is
// read and written once, and that is nearly all of the traffic: at batch 256 x
// 4096 channels x 16 states 142 MB in 36 us, 0.58 of the copy rate.  Two batch
// rows a thread and 40 warps an SM; four rows and 24 warps took 40 us, one row
// and 64 warps 37.
#include "selscan.cuh"

namespace dwp {

namespace {

constexpr int kStepThreads = 128;
constexpr int kStepRows = 2;  // batch rows a thread takes: their loads are all in flight together

// NL neighbouring lanes share a channel, four states each.  kWide: those four
// are one aligned access in A, B, C and the states, and 4 NL is their number.
template <class T, int NL, bool kWide>
__global__ void __launch_bounds__(kStepThreads, 10) scan_step_kernel(ScanStepParams p) {
    constexpr int kCh = kStepThreads / NL;
    pdl_trigger();
    pdl_wait();
    const int nl = threadIdx.x % NL, n0 = nl * 4;
    const uint32_t g = blockIdx.y / p.group_blocks;
    const int64_t cg = int64_t(blockIdx.y % p.group_blocks) * kCh + threadIdx.x / NL;
    const bool own = cg < p.group;
    const int64_t c = int64_t(g) * p.group + (own ? cg : p.group - 1);
    const int64_t b0 = int64_t(blockIdx.x) * kStepRows;

    auto four = [&](auto *x, float(&v)[4]) {
        using E = std::remove_cv_t<std::remove_reference_t<decltype(*x)>>;
        if constexpr (kWide) {
            load_f32<4, E>(v, x + n0);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = n0 + j < p.states ? to_f32<E>(x[n0 + j]) : 0.0f;
        }
    };
    float A[4], h[kStepRows][4], B[kStepRows][4], C[kStepRows][4], d[kStepRows], u[kStepRows], z[kStepRows];
    int64_t slot[kStepRows];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int64_t b = min(b0 + i, p.batch - 1);
        slot[i] = p.slots ? p.slots[b] : b;
    }
    four(p.A + c * p.states, A);
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int64_t b = min(b0 + i, p.batch - 1);
        if (slot[i] < 0 || slot[i] >= p.num_slots) slot[i] = -1;  // a padding row: nothing is read or kept for it
        const int64_t s = slot[i] < 0 ? 0 : slot[i];
        if (p.num_slots > 0) four(p.state + s * p.state_slot + c * p.states, h[i]);
        four(static_cast<const T *>(p.B) + b * p.b_row + g * p.b_group, B[i]);
        four(static_cast<const T *>(p.C) + b * p.c_row + g * p.c_group, C[i]);
        d[i] = to_f32<T>(static_cast<const T *>(p.dt)[b * p.dt_row + c]);
        u[i] = to_f32<T>(static_cast<const T *>(p.u)[b * p.u_row + c]);
        z[i] = p.z ? to_f32<T>(static_cast<const T *>(p.z)[b * p.z_row + c]) : 0.0f;
    }
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, D = p.D ? p.D[c] : 0.0f;
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        float delta = d[i] + bias;
        if (p.softplus) delta = softplus_poly(delta);
        const float x = delta * u[i];
        float y = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[i][j] = fmaf(ex2(delta * (A[j] * kLog2e)), h[i][j], x * B[i][j]);
            y = fmaf(C[i][j], h[i][j], y);
        }
#pragma unroll
        for (int o = NL / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (!own || b0 + i >= p.batch) continue;
        if (slot[i] >= 0) {
            float *to = p.state + slot[i] * p.state_slot + c * p.states;
            if constexpr (kWide) {
                store_f32<4>(to + n0, h[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n0 + j < p.states) to[n0 + j] = h[i][j];
            }
        }
        if (nl == 0) {
            y = fmaf(D, u[i], y);
            if (p.z) y *= silu(z[i]);
            static_cast<T *>(p.out)[(b0 + i) * p.out_row + c] = from_f32<T>(slot[i] < 0 ? 0.0f : y);
        }
    }
}

template <class T, int NL>
cudaError_t step_nl(ScanStepParams p, cudaStream_t s) {
    constexpr int kCh = kStepThreads / NL;
    p.group_blocks = uint32_t((p.group + kCh - 1) / kCh);
    const dim3 grid(uint32_t((p.batch + kStepRows - 1) / kStepRows), uint32_t(p.groups * p.group_blocks));
    if (p.wide && p.states == 4 * NL)
        return launch_pdl(scan_step_kernel<T, NL, true>, grid, dim3(kStepThreads), 0, s, p);
    return launch_pdl(scan_step_kernel<T, NL, false>, grid, dim3(kStepThreads), 0, s, p);
}

template <class T>
cudaError_t step_t(const ScanStepParams &p, cudaStream_t s) {
    if (p.states <= 8) return step_nl<T, 2>(p, s);
    if (p.states <= 16) return step_nl<T, 4>(p, s);
    if (p.states <= 32) return step_nl<T, 8>(p, s);
    if (p.states <= 64) return step_nl<T, 16>(p, s);
    return step_nl<T, 32>(p, s);
}

}  // namespace

cudaError_t launch_selscan_step(dwp_dtype t, const ScanStepParams &p, cudaStream_t s) {
    if (t == DWP_F32) return step_t<float>(p, s);
    if (t == DWP_BF16) return step_t<__nv_bfloat16>(p, s);
    return step_t<__half>(p, s);
}

}  // namespace dwp
