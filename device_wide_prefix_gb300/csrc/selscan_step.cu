// Selective state space scan, the single-token form: each row of a batch
// moves its sequence's state on by one step and reads it out.
#include "selscan.cuh"

namespace dwp {

namespace {

// One token for each row of a batch; NL lanes per channel as above.
template <class T, int NL>
__global__ void __launch_bounds__(kScanThreads) scan_step_kernel(ScanStepParams p) {
    constexpr int kCh = kScanThreads / NL;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, nl = tid % NL, cl = tid / NL;
    const int64_t b = blockIdx.x;
    const uint32_t g = blockIdx.y / p.group_blocks;
    const int64_t cg = int64_t(blockIdx.y % p.group_blocks) * kCh + cl;
    const bool own = cg < p.group;
    const int64_t c = int64_t(g) * p.group + cg;
    T *out = static_cast<T *>(p.out) + b * p.out_row + c;
    const int64_t slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.num_slots) {  // a padding row
        if (own && nl == 0) *out = from_f32<T>(0.0f);
        return;
    }
    float y = 0.0f, u = 0.0f;
    if (own) {
        u = to_f32<T>(static_cast<const T *>(p.u)[b * p.u_row + c]);
        float d = to_f32<T>(static_cast<const T *>(p.dt)[b * p.dt_row + c]);
        if (p.dt_bias) d += p.dt_bias[c];
        if (p.softplus) d = softplus_poly(d);
        float *st = p.state + slot * p.state_slot + c * p.states;
        const T *B = static_cast<const T *>(p.B) + b * p.b_row + g * p.b_group;
        const T *C = static_cast<const T *>(p.C) + b * p.c_row + g * p.c_group;
#pragma unroll
        for (int j = 0; j < kNT; ++j) {
            const int n = nl * kNT + j;
            if (n < p.states) {
                const float a = ex2(d * (p.A[c * p.states + n] * kLog2e));
                const float h = fmaf(a, st[n], d * u * to_f32<T>(B[n]));
                st[n] = h;
                y = fmaf(to_f32<T>(C[n]), h, y);
            }
        }
    }
#pragma unroll
    for (int o = NL / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (own && nl == 0) {
        if (p.D) y = fmaf(p.D[c], u, y);
        if (p.z) y *= silu(to_f32<T>(static_cast<const T *>(p.z)[b * p.z_row + c]));
        *out = from_f32<T>(y);
    }
}

template <class T, int NL>
cudaError_t step_nl(ScanStepParams p, cudaStream_t s) {
    constexpr int kCh = kScanThreads / NL;
    p.group_blocks = uint32_t((p.group + kCh - 1) / kCh);
    const dim3 grid(uint32_t(p.batch), uint32_t(p.groups * p.group_blocks));
    return launch_pdl(scan_step_kernel<T, NL>, grid, dim3(kScanThreads), 0, s, p);
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
