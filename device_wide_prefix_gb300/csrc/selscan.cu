// Selective state space scan over packed rows: forward and the single-token
// form.  Per channel d and state n,
//
//   delta = softplus(dt + dt_bias)          (or dt)
//   h[t]  = exp(delta A[d,n]) h[t-1] + delta u B[t,n]
//   y[t]  = sum_n C[t,n] h[t] + D u;   out = y * silu(z)
//
// The recurrence runs in registers: a thread owns kNT states of a channel,
// NL neighbouring lanes own all states of it, and the rows go by in tiles of
// kScanTile staged through shared memory.
#include "selscan.cuh"

namespace dwp {

namespace {

template <class T, int NL>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(ScanParams p) {
    constexpr int kCh = kScanThreads / NL;  // channels of a block
    constexpr int kNP = NL * kNT;           // states, padded
    extern __shared__ float4 smem4[];
    float2 *sd = reinterpret_cast<float2 *>(smem4);             // [tile][kCh] (delta, delta u)
    float *sb = reinterpret_cast<float *>(sd + kScanTile * kCh);  // [tile][kNP]
    float *sc = sb + kScanTile * kNP;                           // [tile][kNP]
    float *sy = sc + kScanTile * kNP;                           // [tile][kCh]
    uint32_t *sf = reinterpret_cast<uint32_t *>(sy + kScanTile * kCh);  // [tile]
    pdl_trigger();
    pdl_wait();

    const int tid = threadIdx.x, nl = tid % NL, cl = tid / NL;
    const uint32_t b = blockIdx.x / p.chunks;
    const int64_t t0 = int64_t(blockIdx.x % p.chunks) * p.chunk_rows;
    const int64_t t1 = min(t0 + p.chunk_rows, p.rows);
    const uint32_t g = blockIdx.y / p.group_blocks;
    const int64_t cg = int64_t(blockIdx.y % p.group_blocks) * kCh;  // first channel within the group
    const int64_t cb = int64_t(g) * p.group + cg;
    const int live = int(min(int64_t(kCh), p.group - cg));
    const bool own = cl < live;
    const int64_t c = cb + cl;
    const int n0 = nl * kNT;

    float A2[kNT], h[kNT];
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
        A2[j] = own && n0 + j < p.states ? p.A[c * p.states + n0 + j] * kLog2e : 0.0f;
        h[j] = 0.0f;
    }
    auto load_state = [&](const float *from, int64_t i) {
#pragma unroll
        for (int j = 0; j < kNT; ++j)
            h[j] = from && own && n0 + j < p.states ? from[(i * p.channels + c) * p.states + n0 + j] : 0.0f;
    };
    auto save_state = [&](float *to, int64_t i) {
#pragma unroll
        for (int j = 0; j < kNT; ++j)
            if (own && n0 + j < p.states) to[(i * p.channels + c) * p.states + n0 + j] = h[j];
    };
    if (t0 == 0 && !p.segmap) load_state(p.initial, b);

    const T *u = static_cast<const T *>(p.u) + int64_t(b) * p.u_batch + cb;
    const T *dt = static_cast<const T *>(p.dt) + int64_t(b) * p.dt_batch + cb;
    const T *z = p.z ? static_cast<const T *>(p.z) + int64_t(b) * p.z_batch + cb : nullptr;
    const T *B = static_cast<const T *>(p.B) + int64_t(b) * p.b_batch + g * p.b_group;
    const T *C = static_cast<const T *>(p.C) + int64_t(b) * p.c_batch + g * p.c_group;
    T *out = static_cast<T *>(p.out) + int64_t(b) * p.out_batch + cb;

    for (int64_t s0 = t0; s0 < t1; s0 += kScanTile) {
        const int rows = int(min(int64_t(kScanTile), t1 - s0));
        for (int i = tid; i < rows * kCh; i += kScanThreads) {
            const int r = i / kCh, k = i % kCh;
            float2 v = make_float2(0.0f, 0.0f);
            if (k < live) {
                v.x = to_f32<T>(dt[(s0 + r) * p.dt_row + k]);
                if (p.dt_bias) v.x += p.dt_bias[cb + k];
                if (p.softplus) v.x = softplus(v.x);
                v.y = v.x * to_f32<T>(u[(s0 + r) * p.u_row + k]);
            }
            sd[i] = v;
        }
        for (int i = tid; i < rows * kNP; i += kScanThreads) {
            const int r = i / kNP, n = i % kNP;
            sb[i] = n < p.states ? to_f32<T>(B[(s0 + r) * p.b_row + n]) : 0.0f;
            sc[i] = n < p.states ? to_f32<T>(C[(s0 + r) * p.c_row + n]) : 0.0f;
        }
        if (p.segmap && tid < rows) sf[tid] = p.segmap[s0 + tid];
        __syncthreads();
        if (p.checkpoints) save_state(p.checkpoints, int64_t(b) * p.tiles + s0 / kScanTile);
        for (int r = 0; r < rows; ++r) {
            const uint32_t f = p.segmap ? sf[r] : 0u;
            if (f == kRowOutside) continue;
            if (f & kRowHead) load_state(p.initial, f & kRowSegment);
            const float2 d = sd[r * kCh + cl];
            float y = 0.0f;
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                h[j] = fmaf(ex2(d.x * A2[j]), h[j], d.y * sb[r * kNP + n0 + j]);
                y = fmaf(sc[r * kNP + n0 + j], h[j], y);
            }
#pragma unroll
            for (int o = NL / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
            if (nl == 0) sy[r * kCh + cl] = y;
            if ((f & kRowTail) && p.final) save_state(p.final, f & kRowSegment);
        }
        __syncthreads();
        for (int i = tid; i < rows * kCh; i += kScanThreads) {
            const int r = i / kCh, k = i % kCh;
            if (k >= live || (p.segmap && sf[r] == kRowOutside)) continue;
            float y = sy[i];
            if (p.D) y = fmaf(p.D[cb + k], to_f32<T>(u[(s0 + r) * p.u_row + k]), y);
            if (z) y *= silu(to_f32<T>(z[(s0 + r) * p.z_row + k]));
            out[(s0 + r) * p.out_row + k] = from_f32<T>(y);
        }
        __syncthreads();
    }
    if (!p.segmap && p.final && t1 == p.rows) save_state(p.final, b);
}

// One code word per packed row: its segment, and whether it is the segment's
// first or last row.
__global__ void __launch_bounds__(256)
    segment_map_kernel(const uint32_t *offsets, uint32_t nseg, uint32_t rows, uint32_t *map) {
    pdl_trigger();
    pdl_wait();
    const uint32_t t = blockIdx.x * 256u + threadIdx.x;
    if (t >= rows) return;
    const uint32_t s = segment_of(offsets, nseg, t);
    uint32_t code = kRowOutside;
    if (s < nseg && offsets[s] <= t)
        code = s | (offsets[s] == t ? kRowHead : 0u) | (min(offsets[s + 1], rows) == t + 1u ? kRowTail : 0u);
    map[t] = code;
}

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
        if (p.softplus) d = softplus(d);
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
cudaError_t scan_nl(ScanParams p, cudaStream_t s) {
    constexpr int kCh = kScanThreads / NL;
    p.group_blocks = uint32_t((p.group + kCh - 1) / kCh);
    const size_t smem = sizeof(float) * kScanTile * (3 * kCh + 2 * NL * kNT + 1);
    if (device_blocks(reinterpret_cast<const void *>(scan_kernel<T, NL>), kScanThreads, smem) == 0)
        return cudaErrorInvalidConfiguration;
    const dim3 grid(uint32_t(p.batch * p.chunks), uint32_t(p.groups * p.group_blocks));
    return launch_pdl(scan_kernel<T, NL>, grid, dim3(kScanThreads), smem, s, p);
}

template <class T>
cudaError_t scan_t(const ScanParams &p, cudaStream_t s) {
    if (p.states <= 8) return scan_nl<T, 2>(p, s);
    if (p.states <= 16) return scan_nl<T, 4>(p, s);
    if (p.states <= 32) return scan_nl<T, 8>(p, s);
    if (p.states <= 64) return scan_nl<T, 16>(p, s);
    return scan_nl<T, 32>(p, s);
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

cudaError_t launch_segment_map(const uint32_t *offsets, uint32_t nseg, uint32_t rows, uint32_t *map,
                               cudaStream_t s) {
    return launch_pdl(segment_map_kernel, dim3((rows + 255u) / 256u), dim3(256), 0, s, offsets, nseg, rows, map);
}

cudaError_t launch_selscan(dwp_dtype t, const ScanParams &p, cudaStream_t s) {
    if (t == DWP_F32) return scan_t<float>(p, s);
    if (t == DWP_BF16) return scan_t<__nv_bfloat16>(p, s);
    return scan_t<__half>(p, s);
}

cudaError_t launch_selscan_step(dwp_dtype t, const ScanStepParams &p, cudaStream_t s) {
    if (t == DWP_F32) return step_t<float>(p, s);
    if (t == DWP_BF16) return step_t<__nv_bfloat16>(p, s);
    return step_t<__half>(p, s);
}

}  // namespace dwp
