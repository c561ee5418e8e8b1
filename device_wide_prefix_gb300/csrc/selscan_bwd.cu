// Gradient of the selective state space scan.  With dy = dout * silu(z), per
// channel d and state n, rows from last to first:
//
//   dh[t] = C[t,n] dy[t] + a[t+1] dh[t+1]        (a = exp(delta A))
//   dC[t,n] = sum_d dy h[t],   dB[t,n] = sum_d dh delta u
//   q1 = sum_n dh B,           q2 = sum_n dh a h[t-1] A
//   du = delta q1 + D dy,      ddelta = u q1 + q2
//   dA = sum_t dh a h[t-1] delta
//
// The states come again from those the forward kept before every kCheckpointRows
// rows: a tile is first walked forward to its kSub-row boundaries, then each
// kSub rows are walked forward once more with the states kept in registers
// and backward.
#include "selscan.cuh"

namespace dwp {

namespace {

constexpr int kSub = 8;
constexpr int kSubs = kCheckpointRows / kSub;

template <class T, int NL>
__global__ void __launch_bounds__(kScanThreads) scan_backward_kernel(ScanBackwardParams q) {
    constexpr int kCh = kScanThreads / NL;
    constexpr int kNP = NL * kNT;
    constexpr int kWarps = kScanThreads / 32;
    const ScanParams &p = q.f;
    extern __shared__ float4 smem4[];
    float2 *sd = reinterpret_cast<float2 *>(smem4);               // (delta, delta u)
    float *sg = reinterpret_cast<float *>(sd + kCheckpointRows * kCh);  // dy
    float *s1 = sg + kCheckpointRows * kCh;                             // q1
    float *s2 = s1 + kCheckpointRows * kCh;                             // q2
    float *sy = s2 + kCheckpointRows * kCh;                             // y
    float *sb = sy + kCheckpointRows * kCh;
    float *sc = sb + kCheckpointRows * kNP;
    float *sr = sc + kCheckpointRows * kNP;                             // [warp][kSub][2 kNP]
    uint32_t *sf = reinterpret_cast<uint32_t *>(sr + kWarps * kSub * 2 * kNP);
    pdl_trigger();
    pdl_wait();

    const int tid = threadIdx.x, nl = tid % NL, cl = tid / NL, warp = tid / 32, lane = tid % 32;
    const uint32_t b = blockIdx.x / p.chunks;
    const int64_t t0 = int64_t(blockIdx.x % p.chunks) * p.chunk_rows;
    const int64_t t1 = min(t0 + p.chunk_rows, p.rows);
    const uint32_t g = blockIdx.y / p.group_blocks, gb = blockIdx.y % p.group_blocks;
    const int64_t cg = int64_t(gb) * kCh;
    const int64_t cb = int64_t(g) * p.group + cg;
    const int live = int(min(int64_t(kCh), p.group - cg));
    const bool own = cl < live;
    const int64_t c = cb + cl;
    const int n0 = nl * kNT;

    float A[kNT], e[kNT], dA[kNT], h[kNT];
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
        A[j] = own && n0 + j < p.states ? p.A[c * p.states + n0 + j] : 0.0f;
        e[j] = dA[j] = 0.0f;
    }
    auto load_state = [&](float(&v)[kNT], const float *from, int64_t i) {
#pragma unroll
        for (int j = 0; j < kNT; ++j)
            v[j] = from && own && n0 + j < p.states ? from[(i * p.channels + c) * p.states + n0 + j] : 0.0f;
    };
    auto save_state = [&](float *to, int64_t i, const float(&v)[kNT]) {
#pragma unroll
        for (int j = 0; j < kNT; ++j)
            if (own && n0 + j < p.states) to[(i * p.channels + c) * p.states + n0 + j] = v[j];
    };
    if (!p.segmap && t1 == p.rows) load_state(e, q.grad_final, b);

    const T *u = static_cast<const T *>(p.u) + int64_t(b) * p.u_batch + cb;
    const T *dt = static_cast<const T *>(p.dt) + int64_t(b) * p.dt_batch + cb;
    const T *z = p.z ? static_cast<const T *>(p.z) + int64_t(b) * p.z_batch + cb : nullptr;
    const T *B = static_cast<const T *>(p.B) + int64_t(b) * p.b_batch + g * p.b_group;
    const T *C = static_cast<const T *>(p.C) + int64_t(b) * p.c_batch + g * p.c_group;
    const T *go = static_cast<const T *>(q.grad_out) + int64_t(b) * q.grad_batch + cb;
    // gradients of the inputs are dense
    const int64_t out0 = int64_t(b) * p.rows * p.channels + cb;
    T *gu = static_cast<T *>(q.grad_u) + out0, *gdt = static_cast<T *>(q.grad_dt) + out0;
    T *gz = q.grad_z ? static_cast<T *>(q.grad_z) + out0 : nullptr;
    float acc_D = 0.0f, acc_bias = 0.0f;  // of channel tid % kCh

    const int64_t last = t0 + (t1 - 1 - t0) / kCheckpointRows * kCheckpointRows;
    for (int64_t s0 = last; s0 >= t0; s0 -= kCheckpointRows) {
        const int rows = int(min(int64_t(kCheckpointRows), t1 - s0));
        for (int i = tid; i < kCheckpointRows * kCh; i += kScanThreads) {
            const int r = i / kCh, k = i % kCh;
            float2 v = make_float2(0.0f, 0.0f);
            float dy = 0.0f;
            if (k < live && r < rows) {
                v.x = to_f32<T>(dt[(s0 + r) * p.dt_row + k]);
                if (p.dt_bias) v.x += p.dt_bias[cb + k];
                if (p.softplus) v.x = softplus_poly(v.x);
                v.y = v.x * to_f32<T>(u[(s0 + r) * p.u_row + k]);
                dy = to_f32<T>(go[(s0 + r) * q.grad_row + k]);
                if (z) dy *= silu(to_f32<T>(z[(s0 + r) * p.z_row + k]));
            }
            sd[i] = v;
            sg[i] = dy;
        }
        for (int i = tid; i < kCheckpointRows * kNP; i += kScanThreads) {
            const int r = i / kNP, n = i % kNP;
            sb[i] = r < rows && n < p.states ? to_f32<T>(B[(s0 + r) * p.b_row + n]) : 0.0f;
            sc[i] = r < rows && n < p.states ? to_f32<T>(C[(s0 + r) * p.c_row + n]) : 0.0f;
        }
        if (tid < kCheckpointRows) sf[tid] = tid >= rows ? kRowOutside : p.segmap ? p.segmap[s0 + tid] : 0u;
        __syncthreads();

        load_state(h, p.checkpoints, int64_t(b) * p.tiles + s0 / kCheckpointRows);
        auto step = [&](int r) {  // the state past row r
            const uint32_t f = sf[r];
            if (f == kRowOutside) return;
            if (f & kRowHead) load_state(h, p.initial, f & kRowSegment);
            const float2 d = sd[r * kCh + cl];
#pragma unroll
            for (int j = 0; j < kNT; ++j)
                h[j] = fmaf(ex2(d.x * (A[j] * kLog2e)), h[j], d.y * sb[r * kNP + n0 + j]);
        };
        float at[kSubs][kNT];  // states before each kSub rows
#pragma unroll
        for (int k = 0; k < kSubs; ++k) {
#pragma unroll
            for (int j = 0; j < kNT; ++j) at[k][j] = h[j];
            if (k < kSubs - 1)
                for (int r = 0; r < kSub; ++r) step(k * kSub + r);
        }
#pragma unroll
        for (int k = kSubs - 1; k >= 0; --k) {
            float hist[kSub][kNT];  // states before each row
#pragma unroll
            for (int j = 0; j < kNT; ++j) h[j] = at[k][j];
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const int r = k * kSub + i;
                const uint32_t f = sf[r];
                if (f != kRowOutside && (f & kRowHead)) load_state(h, p.initial, f & kRowSegment);
#pragma unroll
                for (int j = 0; j < kNT; ++j) hist[i][j] = h[j];
                if (f == kRowOutside) continue;
                const float2 d = sd[r * kCh + cl];
                float y = 0.0f;
#pragma unroll
                for (int j = 0; j < kNT; ++j) {
                    h[j] = fmaf(ex2(d.x * (A[j] * kLog2e)), h[j], d.y * sb[r * kNP + n0 + j]);
                    y = fmaf(sc[r * kNP + n0 + j], h[j], y);
                }
#pragma unroll
                for (int o = NL / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (nl == 0) sy[r * kCh + cl] = y;
            }
#pragma unroll
            for (int i = kSub - 1; i >= 0; --i) {
                const int r = k * kSub + i;
                const uint32_t f = sf[r];
                if (f == kRowOutside) continue;
                if (f & kRowTail) load_state(e, q.grad_final, f & kRowSegment);
                const float2 d = sd[r * kCh + cl];
                const float dy = sg[r * kCh + cl];
                float q1 = 0.0f, q2 = 0.0f, db[kNT], dc[kNT];
#pragma unroll
                for (int j = 0; j < kNT; ++j) {
                    const float bn = sb[r * kNP + n0 + j];
                    const float a = ex2(d.x * (A[j] * kLog2e));
                    const float dh = fmaf(dy, sc[r * kNP + n0 + j], e[j]);
                    dc[j] = dy * fmaf(a, hist[i][j], d.y * bn);
                    db[j] = dh * d.y;
                    q1 = fmaf(dh, bn, q1);
                    e[j] = dh * a;
                    const float w = e[j] * hist[i][j];
                    q2 = fmaf(w, A[j], q2);
                    dA[j] = fmaf(w, d.x, dA[j]);
                }
                if (f & kRowHead) {
                    if (q.grad_initial) save_state(q.grad_initial, f & kRowSegment, e);
#pragma unroll
                    for (int j = 0; j < kNT; ++j) e[j] = 0.0f;
                }
#pragma unroll
                for (int o = NL / 2; o > 0; o >>= 1) {
                    q1 += __shfl_xor_sync(0xffffffffu, q1, o);
                    q2 += __shfl_xor_sync(0xffffffffu, q2, o);
                }
                if (nl == 0) s1[r * kCh + cl] = q1, s2[r * kCh + cl] = q2;
#pragma unroll
                for (int j = 0; j < kNT; ++j) {
#pragma unroll
                    for (int o = NL; o < 32; o <<= 1) {
                        db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
                        dc[j] += __shfl_xor_sync(0xffffffffu, dc[j], o);
                    }
                    if (lane < NL) {
                        float *to = sr + (warp * kSub + i) * 2 * kNP + n0 + j;
                        to[0] = db[j];
                        to[kNP] = dc[j];
                    }
                }
            }
            __syncthreads();
            for (int i = tid; i < kSub * 2 * kNP; i += kScanThreads) {
                const int r = k * kSub + i / (2 * kNP), n = i % kNP, which = i / kNP % 2;
                if (sf[r] == kRowOutside || n >= p.states) continue;
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += sr[w * kSub * 2 * kNP + i];
                q.partial_bc[(((int64_t(gb) * p.batch + b) * p.rows + s0 + r) * p.groups + g) * 2 * p.states +
                             which * p.states + n] = s;
            }
            __syncthreads();
        }
        for (int i = tid; i < rows * kCh; i += kScanThreads) {
            const int r = i / kCh, k = i % kCh;
            if (k >= live || sf[r] == kRowOutside) continue;
            const int64_t t = s0 + r;
            const float uv = to_f32<T>(u[t * p.u_row + k]);
            const float Dv = p.D ? p.D[cb + k] : 0.0f;
            float raw = to_f32<T>(dt[t * p.dt_row + k]);
            if (p.dt_bias) raw += p.dt_bias[cb + k];
            const float q1 = s1[i], dy = sg[i];
            float dd = fmaf(q1, uv, s2[i]);
            if (p.softplus) dd *= sigmoid(raw);
            gu[t * p.channels + k] = from_f32<T>(fmaf(q1, sd[i].x, Dv * dy));
            gdt[t * p.channels + k] = from_f32<T>(dd);
            if (z) {
                const float zv = to_f32<T>(z[t * p.z_row + k]);
                gz[t * p.channels + k] =
                    from_f32<T>(to_f32<T>(go[t * q.grad_row + k]) * fmaf(Dv, uv, sy[i]) * silu_slope(zv));
            }
            acc_D = fmaf(dy, uv, acc_D);
            acc_bias += dd;
        }
        __syncthreads();
    }
    if (!p.segmap && t0 == 0 && q.grad_initial) save_state(q.grad_initial, b, e);

    // the parameters' shares of this block: [dA | dD | ddt_bias]
    float *part = q.partial + int64_t(blockIdx.x) * p.channels * (p.states + 2);
    save_state(part, 0, dA);
    s1[tid] = acc_D;
    s2[tid] = acc_bias;
    __syncthreads();
    if (tid < live) {
        float d = 0.0f, bias = 0.0f;
        for (int k = tid; k < kScanThreads; k += kCh) d += s1[k], bias += s2[k];
        part[p.channels * p.states + cb + tid] = d;
        part[p.channels * (p.states + 1) + cb + tid] = bias;
    }
}

// dB and dC: the shares of a group's channel blocks, added in order.
template <class T>
__global__ void __launch_bounds__(256) join_bc_kernel(ScanBackwardParams q, int64_t total) {
    pdl_trigger();
    pdl_wait();
    const ScanParams &p = q.f;
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= total) return;
    const int64_t per = int64_t(2) * p.groups * p.states;
    const int64_t row = i / per;
    if (p.segmap && p.segmap[row] == kRowOutside) return;
    float s = 0.0f;
    for (uint32_t k = 0; k < p.group_blocks; ++k) s += q.partial_bc[k * total + i];
    const int64_t at = i % per, g = at / (2 * p.states), which = at / p.states % 2, n = at % p.states;
    T *to = static_cast<T *>(which ? q.grad_C : q.grad_B);
    to[(row * p.groups + g) * p.states + n] = from_f32<T>(s);
}

template <class T, int NL>
cudaError_t backward_nl(ScanBackwardParams q, cudaStream_t s) {
    constexpr int kCh = kScanThreads / NL, kNP = NL * kNT;
    ScanParams &p = q.f;
    p.group_blocks = uint32_t((p.group + kCh - 1) / kCh);
    const size_t smem =
        sizeof(float) * (kCheckpointRows * (6 * kCh + 2 * kNP + 1) + kScanThreads / 32 * kSub * 2 * kNP);
    if (device_blocks(reinterpret_cast<const void *>(scan_backward_kernel<T, NL>), kScanThreads, smem) == 0)
        return cudaErrorInvalidConfiguration;
    const dim3 grid(uint32_t(p.batch * p.chunks), uint32_t(p.groups * p.group_blocks));
    cudaError_t err = launch_pdl(scan_backward_kernel<T, NL>, grid, dim3(kScanThreads), smem, s, q);
    if (err != cudaSuccess) return err;
    const int64_t total = int64_t(p.batch) * p.rows * p.groups * 2 * p.states;
    return launch_pdl(join_bc_kernel<T>, dim3(uint32_t((total + 255) / 256)), dim3(256), 0, s, q, total);
}

template <class T>
cudaError_t backward_t(const ScanBackwardParams &q, cudaStream_t s) {
    const int n = q.f.states;
    if (n <= 8) return backward_nl<T, 2>(q, s);
    if (n <= 16) return backward_nl<T, 4>(q, s);
    if (n <= 32) return backward_nl<T, 8>(q, s);
    if (n <= 64) return backward_nl<T, 16>(q, s);
    return backward_nl<T, 32>(q, s);
}

}  // namespace

int64_t scan_block_channels(int64_t states) {
    const int nl = states <= 8 ? 2 : states <= 16 ? 4 : states <= 32 ? 8 : states <= 64 ? 16 : 32;
    return kScanThreads / nl;
}

cudaError_t launch_selscan_backward(dwp_dtype t, const ScanBackwardParams &q, cudaStream_t s) {
    if (t == DWP_F32) return backward_t<float>(q, s);
    if (t == DWP_BF16) return backward_t<__nv_bfloat16>(q, s);
    return backward_t<__half>(q, s);
}

}  // namespace dwp
