// Selective state space scan over packed rows, forward.  Per channel d and
// state n,
//
//   delta = softplus(dt + dt_bias)          (or dt)
//   h[t]  = exp(delta A[d,n]) h[t-1] + delta u B[t,n]
//   y[t]  = sum_n C[t,n] h[t] + D u;   out = y * silu(z)
//
// The recurrence runs in registers, and a block is one warp that walks its
// channels through all of its rows.  A lane owns NT states of two neighbouring
// channels (NL lanes share a pair of channels with more states than that), so
// loading, softplus, the gate and storing need no other lane; only B and C,
// which every channel shares, go through shared memory.
//
// Long sequences are cut into chunks of rows for more warps: a first pass
// walks every chunk but the last from a zero state and keeps its last state
// and the sum of delta (the product of a chunk's decays is exp(A sum delta)),
// a short kernel carries the states from chunk to chunk, and the second pass
// walks every chunk from its true first state.
//
// What bounds it: per state update 4 multiply-adds' worth of f32 work and one
// exponential (4 cycles a warp each way), and per row and channel about 45
// instructions of softplus, gate and accesses, a third of the whole at 16
// states.  8192 rows x 4096 channels x 16 states bf16: 295 us (first pass 120,
// second 172), issue 0.61-0.64 a cycle at 2.4 to 2.6 warps a scheduler.  Packed
// f32 instructions keep the rate of the scalar ones in half the issue slots.
// Fewer registers for more warps lost (one channel a lane 331 us; 128 registers
// 430), so did more rows in flight a lane (four 324, one 356, two 294).
#pragma once

#include "selscan.cuh"

namespace dwp {

namespace {

constexpr int kAhead = 2;  // rows loaded ahead of their use

// Two neighbouring channels of a row, as loaded: the bits are taken apart at
// their first use only, so that a load is waited for there and not before.
template <class T>
struct Two {
    uint32_t bits;
    __device__ __forceinline__ float2 f32() const {
        const Pack<T, 2> v = *reinterpret_cast<const Pack<T, 2> *>(&bits);
        return make_float2(to_f32<T>(v.e[0]), to_f32<T>(v.e[1]));
    }
    __device__ __forceinline__ void load(const T *p) { bits = *reinterpret_cast<const uint32_t *>(p); }
    __device__ __forceinline__ void load(const T *p, const T *q) {
        const auto *a = reinterpret_cast<const uint16_t *>(p), *b = reinterpret_cast<const uint16_t *>(q);
        bits = uint32_t(*a) | uint32_t(*b) << 16;
    }
};
template <>
struct Two<float> {
    float2 v;
    __device__ __forceinline__ float2 f32() const { return v; }
    __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const float2 *>(p); }
    __device__ __forceinline__ void load(const float *p, const float *q) { v = make_float2(*p, *q); }
};

// What a walk computes.  kWalkOut: the scan.  kWalkStates: the first pass
// over chunks, last states and sums of delta only.  kWalkBack: the same for
// the gradient, whose recurrence runs from the last row to the first:
// e = exp(delta A) (e + dout silu(z) C), with u standing for dout, B for C,
// initial for the final state's gradient, and a segment's last row in the
// place of its first.
enum : int { kWalkStates = 0, kWalkOut = 1, kWalkBack = 2 };

// kWide: two neighbouring channels, and four neighbouring states of B and C,
// are one aligned access, so that the loads are straight code: a load under a
// branch is waited for where the branch ends, and the rows ahead of their use
// would buy nothing.
template <class T, int NT, int NL, int kMode, bool kWide>
__global__ void __launch_bounds__(32, 10) selscan_kernel(ScanParams p) {
    constexpr int kC = 64 / NL, kN = NT * NL, kP = NT / 2;
    constexpr int kRows = kN <= 16 ? 16 : kN <= 32 ? 8 : 4;  // rows of B and C staged at once
    static_assert(kRows % (2 * kAhead) == 0 && kCheckpointRows % kRows == 0, "");
    __shared__ float4 bc4[2][kRows * 2 * kN / 4];  // B, then C, of each row
    const int lane = threadIdx.x, nl = lane % NL, n0 = nl * NT;
    pdl_trigger();
    pdl_wait();

    constexpr bool kOut = kMode == kWalkOut, kBack = kMode == kWalkBack, kGate = kMode != kWalkStates;
    constexpr uint32_t kFirst = kBack ? kRowTail : kRowHead;
    const uint32_t chunks = kOut ? uint32_t(p.chunks) : uint32_t(p.chunks - 1);
    const uint32_t b = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int64_t t0 = int64_t(kBack ? uint32_t(p.chunks) - 1u - chunk : chunk) * p.chunk_rows;
    const int64_t t1 = min(t0 + p.chunk_rows, p.rows);
    const uint32_t g = blockIdx.y / p.group_blocks;
    const int64_t cg = int64_t(blockIdx.y % p.group_blocks) * kC;  // first channel within the group
    const int64_t cb = int64_t(g) * p.group + cg;
    const int live = int(min(int64_t(kC), p.group - cg));
    // Where the lane loads: its channels, or live ones in place of those past
    // the last, so that no load needs a predicate.  One access for both
    // channels: live is even, and so is every first channel.
    const int ch = lane / NL * 2;
    const uint32_t c0 = uint32_t(min(ch, kWide ? live - 2 : live - 1)), c1 = uint32_t(min(ch + 1, live - 1));

    F2 A2[2][kP], h[2][kP];
    const bool whole = p.states == kN && p.states_wide;  // every lane's states are live, in 16-byte pieces
    auto load_states = [&](F2(&v)[2][kP], const float *from, int64_t i) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float *x = from + (i * p.channels + cb + min(ch + c, live - 1)) * p.states + n0;
            if (whole) {
#pragma unroll
                for (int j = 0; j < kP; j += 2) {
                    const float4 q = reinterpret_cast<const float4 *>(x)[j / 2];
                    v[c][j] = f2(q.x, q.y), v[c][j + 1] = f2(q.z, q.w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kP; ++j)
                    v[c][j] = f2(n0 + 2 * j < p.states ? x[2 * j] : 0.0f, n0 + 2 * j + 1 < p.states ? x[2 * j + 1] : 0.0f);
            }
        }
    };
    auto load_state = [&](const float *from, int64_t i) {
        if (from) {
            load_states(h, from, i);
        } else {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < kP; ++j) h[c][j] = f2(0.0f, 0.0f);
        }
    };
    auto save_state = [&](float *to, int64_t i) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (ch + c >= live) continue;
            float *x = to + (i * p.channels + cb + ch + c) * p.states + n0;
#pragma unroll
            for (int j = 0; j < kP; j += 2) {
                const float2 lo = unpack(h[c][j]), hi = unpack(h[c][j + 1]);
                if (whole) {
                    reinterpret_cast<float4 *>(x)[j / 2] = make_float4(lo.x, lo.y, hi.x, hi.y);
                } else {
                    if (n0 + 2 * j < p.states) x[2 * j] = lo.x;
                    if (n0 + 2 * j + 1 < p.states) x[2 * j + 1] = lo.y;
                    if (n0 + 2 * j + 2 < p.states) x[2 * j + 2] = hi.x;
                    if (n0 + 2 * j + 3 < p.states) x[2 * j + 3] = hi.y;
                }
            }
        }
    };
    load_states(A2, p.A, 0);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < kP; ++j) A2[c][j] = decay_rate(A2[c][j]);
    if (kOut && chunk > 0) load_state(p.carry, int64_t(b) * (p.chunks - 1) + chunk - 1);
    else load_state(!p.segmap && chunk == 0 ? p.initial : nullptr, b);

    const T *u = static_cast<const T *>(p.u) + int64_t(b) * p.u_batch + cb;
    const T *dt = static_cast<const T *>(p.dt) + int64_t(b) * p.dt_batch + cb;
    auto place = [&](int64_t s) { return kBack ? t0 + t1 - 1 - s : s; };  // the row that the walk meets as row s
    const bool gate = kGate && p.z;
    const T *z = gate ? static_cast<const T *>(p.z) + int64_t(b) * p.z_batch + cb : u;
    const int64_t z_row = gate ? p.z_row : p.u_row;
    const T *B = static_cast<const T *>(p.B) + int64_t(b) * p.b_batch + g * p.b_group;
    const T *C = static_cast<const T *>(p.C) + int64_t(b) * p.c_batch + g * p.c_group;
    T *out = static_cast<T *>(p.out) + int64_t(b) * p.out_batch + cb;
    const uint32_t *map = p.segmap;
    float2 bias = make_float2(0.0f, 0.0f), Dv = make_float2(0.0f, 0.0f);
    if (p.dt_bias) bias = make_float2(p.dt_bias[cb + c0], p.dt_bias[cb + c1]);
    if (p.D) Dv = make_float2(p.D[cb + c0], p.D[cb + c1]);

    // B and C of kRows rows as f32; states past the last are 0
    constexpr int kPieces = kRows * kN / 4, kEach = (kPieces + 31) / 32;
    Pack<T, 4> rb[kEach], rc[kEach];
    auto fetch = [&](int64_t s0) {  // rows past the last are read as the last
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int q = lane + 32 * i, r = q / (kN / 4), n = q % (kN / 4) * 4;
            const int64_t t = place(min(s0 + r, t1 - 1));
            if constexpr (kWide) {
                const int m = min(n, p.states - 4);
                rb[i] = *reinterpret_cast<const Pack<T, 4> *>(B + t * p.b_row + m);
                if (kOut) rc[i] = *reinterpret_cast<const Pack<T, 4> *>(C + t * p.c_row + m);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int m = min(n + j, p.states - 1);
                    rb[i].e[j] = B[t * p.b_row + m];
                    if (kOut) rc[i].e[j] = C[t * p.c_row + m];
                }
            }
        }
    };
    auto keep = [&](int k) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int q = lane + 32 * i, r = q / (kN / 4), n = q % (kN / 4);
            if (kPieces % 32 != 0 && q >= kPieces) break;
            float fb[4], fc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool ok = 4 * n + j < p.states;
                fb[j] = ok ? to_f32<T>(rb[i].e[j]) : 0.0f;
                fc[j] = kOut && ok ? to_f32<T>(rc[i].e[j]) : 0.0f;
            }
            float4 *to = bc4[k] + r * (kN / 2) + n;
            to[0] = make_float4(fb[0], fb[1], fb[2], fb[3]);
            if (kOut) to[kN / 4] = make_float4(fc[0], fc[1], fc[2], fc[3]);
        }
    };

    float2 sum = make_float2(0.0f, 0.0f);  // of delta, in the first pass
    bool head_seen = false;

    // Groups of kAhead rows pass through three stages: loaded, converted
    // (delta and delta u), stepped and written.  One turn converts the next
    // group, loads the one after it and steps the current one, so that the
    // chains of each stage fill the others' waits.
    struct Raw {
        Two<T> dt[kAhead], u[kAhead], z[kAhead];
    } raw;
    struct Ready {
        float d[2][kAhead], x[2][kAhead];
        Two<T> u[kAhead], z[kAhead];
    } even, odd;
    T *out_at = out + t0 * p.out_row;
    auto load = [&](int64_t s) {  // rows past the last are read as the last
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t t = place(min(s + i, t1 - 1));
            const T *pd = dt + t * p.dt_row, *pu = u + t * p.u_row, *pz = z + t * z_row;
            if constexpr (kWide) {
                raw.dt[i].load(pd + c0);
                raw.u[i].load(pu + c0);
                if (kGate) raw.z[i].load(pz + c0);
            } else {
                raw.dt[i].load(pd + c0, pd + c1);
                raw.u[i].load(pu + c0, pu + c1);
                if (kGate) raw.z[i].load(pz + c0, pz + c1);
            }
        }
    };
    // Ask L2 for rows that are loaded kRows rows later: the registers hold too
    // few rows in flight to cover the way from HBM.
    auto prefetch = [&](int64_t s) {
        if (s + kRows > t1) return;
        const int64_t t = place(s + lane % kRows);
        if (kRows == 16) {
            prefetch_l2(lane < 16 ? dt + t * p.dt_row : u + t * p.u_row);
            if (kGate && lane < 16) prefetch_l2(z + t * z_row);
        }
    };
    auto convert = [&](Ready &to) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            float2 d = raw.dt[i].f32();
            const float2 uv = raw.u[i].f32();
            d.x += bias.x, d.y += bias.y;
            if (p.softplus) d.x = softplus_poly(d.x), d.y = softplus_poly(d.y);
            to.d[0][i] = d.x, to.d[1][i] = d.y;
            if constexpr (kBack) {
                to.x[0][i] = uv.x, to.x[1][i] = uv.y;
                if (gate) {
                    const float2 zv = raw.z[i].f32();
                    to.x[0][i] *= silu(zv.x), to.x[1][i] *= silu(zv.y);
                }
            } else {
                to.x[0][i] = d.x * uv.x, to.x[1][i] = d.y * uv.y;
            }
            to.u[i] = raw.u[i], to.z[i] = raw.z[i];
        }
    };
    // the states' step of row i of the group; y: this lane's part of C h
    auto step = [&](const Ready &in, int i, const float4 *bc, float (&y)[2]) {
        F2 acc[2];
#pragma unroll
        for (int j = 0; j < kP; j += 2) {
            const float4 bq = bc[(n0 + 2 * j) / 4];
            const F2 Bv[2] = {f2(bq.x, bq.y), f2(bq.z, bq.w)};
            F2 Cv[2];
            if (kOut) {
                const float4 cq = bc[(kN + n0 + 2 * j) / 4];
                Cv[0] = f2(cq.x, cq.y), Cv[1] = f2(cq.z, cq.w);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float2 e = unpack(mul2(f2(in.d[c][i], in.d[c][i]), A2[c][j + q]));
                    const F2 a = f2(ex2(e.x), ex2(e.y)), x = f2(in.x[c][i], in.x[c][i]);
                    h[c][j + q] = kBack ? mul2(a, fma2(x, Bv[q], h[c][j + q])) : fma2(a, h[c][j + q], mul2(x, Bv[q]));
                    if (kOut) acc[c] = j + q == 0 ? mul2(Cv[q], h[c][0]) : fma2(Cv[q], h[c][j + q], acc[c]);
                }
        }
        if (kOut) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float2 v = unpack(acc[c]);
                y[c] = v.x + v.y;
            }
        } else {
            sum.x += in.d[0][i], sum.y += in.d[1][i];
        }
    };

    int k = 0, rows = 0;     // the tile's buffer and rows
    uint32_t code = 0u;      // of row `lane` of the tile
    bool plain = true;       // no row of the tile needs a look
    // rows r .. r + kAhead of the tile at s0, from `now`; `next` is made ready
    auto turn = [&](int64_t s0, int r, const Ready &now, Ready &next) {
        convert(next);
        load(s0 + r + 2 * kAhead);
        const float4 *bc = bc4[k] + r * (kN / 2);
        float y[kAhead][2] = {};
        uint32_t skip = 0u;  // rows that are not written
        if (plain && r + kAhead <= rows) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) step(now, i, bc + i * (kN / 2), y[i]);
        } else {
            Ready one = now;  // row i at place 0: the rows go by one at a time
#pragma unroll 1
            for (int i = 0; i < kAhead; ++i) {
                const uint32_t f = r + i < rows ? __shfl_sync(0xffffffffu, code, r + i) : kRowOutside;
                float v[2] = {0.0f, 0.0f};
                if (f == kRowOutside) {
                    skip |= 1u << i;
                } else {
                    if (f & kFirst) {
                        load_state(p.initial, f & kRowSegment);
                        head_seen = true;
                    }
                    step(one, 0, bc + i * (kN / 2), v);
                    if (kOut && (f & kRowTail) && p.final) save_state(p.final, f & kRowSegment);
                }
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    if (q + 1 < kAhead) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) one.d[c][q] = one.d[c][q + 1], one.x[c][q] = one.x[c][q + 1];
                    }
                    if (q == i) y[q][0] = v[0], y[q][1] = v[1];
                }
            }
        }
        if (kOut) {
#pragma unroll
            for (int o = 1; o < NL; o <<= 1)
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    y[i][0] += __shfl_xor_sync(0xffffffffu, y[i][0], o);
                    y[i][1] += __shfl_xor_sync(0xffffffffu, y[i][1], o);
                }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float2 uv = now.u[i].f32();
                y[i][0] = fmaf(Dv.x, uv.x, y[i][0]), y[i][1] = fmaf(Dv.y, uv.y, y[i][1]);
                if (gate) {
                    const float2 zv = now.z[i].f32();
                    y[i][0] *= silu(zv.x), y[i][1] *= silu(zv.y);
                }
            }
            if ((NL == 1 || nl == 0) && ch < live) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (skip >> i & 1u) continue;
                    T *to = out_at + i * p.out_row + ch;
                    if constexpr (kWide) {
                        store_f32<2>(to, y[i]);
                    } else {
                        to[0] = from_f32<T>(y[i][0]);
                        if (ch + 1 < live) to[1] = from_f32<T>(y[i][1]);
                    }
                }
            }
            out_at += kAhead * p.out_row;
        }
    };

    fetch(t0);
    load(t0);
    convert(even);
    load(t0 + kAhead);
    prefetch(t0 + kRows);
    keep(0);
    __syncwarp();
    for (int64_t s0 = t0; s0 < t1; s0 += kRows, k ^= 1) {
        rows = int(min(int64_t(kRows), t1 - s0));
        if (s0 + kRows < t1) fetch(s0 + kRows);
        prefetch(s0 + 2 * kRows);
        if (map) {  // heads, tails and rows outside need a look
            code = lane < rows ? map[place(s0 + lane)] : 0u;
            plain = __all_sync(0xffffffffu, (code & (kRowHead | kRowTail)) == 0u);
        }
        if (kOut && p.checkpoints && s0 % kCheckpointRows == 0)
            save_state(p.checkpoints, int64_t(b) * p.tiles + s0 / kCheckpointRows);
#pragma unroll 1
        for (int r = 0; r < rows; r += 2 * kAhead) {
            turn(s0, r, even, odd);
            turn(s0, r + kAhead, odd, even);
        }
        if (s0 + kRows < t1) keep(k ^ 1);
        __syncwarp();
    }
    if (kOut) {
        if (!map && p.final && t1 == p.rows) save_state(p.final, b);
    } else {
        const int64_t i = int64_t(b) * (p.chunks - 1) + chunk;
        save_state(p.carry, i);
        if (nl == 0) {
            if (ch < live) p.carry_sum[i * p.channels + cb + ch] = sum.x;
            if (ch + 1 < live) p.carry_sum[i * p.channels + cb + ch + 1] = sum.y;
        }
        if (blockIdx.y == 0 && lane == 0) p.carry_head[i] = head_seen ? 1u : 0u;
    }
}

template <class T, int NT, int NL, bool kWide>
cudaError_t scan_v(ScanParams p, cudaStream_t s) {
    constexpr int kC = 64 / NL;
    p.group_blocks = uint32_t((p.group + kC - 1) / kC);
    const uint32_t units = uint32_t(p.groups * p.group_blocks);
    if (p.chunks > 1) {
        cudaError_t err = launch_pdl(selscan_kernel<T, NT, NL, kWalkStates, kWide>,
                                     dim3(uint32_t(p.batch * (p.chunks - 1)), units), dim3(32), 0, s, p);
        if (err != cudaSuccess) return err;
        err = launch_carry(p, s);
        if (err != cudaSuccess) return err;
    }
    return launch_pdl(selscan_kernel<T, NT, NL, kWalkOut, kWide>, dim3(uint32_t(p.batch * p.chunks), units), dim3(32), 0, s,
                      p);
}

template <class T, int NT, int NL>
cudaError_t scan_w(const ScanParams &p, cudaStream_t s) {
    return p.wide ? scan_v<T, NT, NL, true>(p, s) : scan_v<T, NT, NL, false>(p, s);
}

template <class T>
cudaError_t scan_t(const ScanParams &p, cudaStream_t s) {
    if (p.states <= 8) return scan_w<T, 8, 1>(p, s);
    if (p.states <= 16) return scan_w<T, 16, 1>(p, s);
    if (p.states <= 32) return scan_w<T, 16, 2>(p, s);
    if (p.states <= 64) return scan_w<T, 16, 4>(p, s);
    return scan_w<T, 16, 8>(p, s);
}

// The walk back over all chunks but the first, and the carry over them.
template <class T, int NT, int NL>
cudaError_t back_w(ScanParams p, cudaStream_t s) {
    constexpr int kC = 64 / NL;
    p.group_blocks = uint32_t((p.group + kC - 1) / kC);
    const dim3 grid(uint32_t(p.batch * (p.chunks - 1)), uint32_t(p.groups * p.group_blocks));
    const cudaError_t err =
        p.wide ? launch_pdl(selscan_kernel<T, NT, NL, kWalkBack, true>, grid, dim3(32), 0, s, p)
               : launch_pdl(selscan_kernel<T, NT, NL, kWalkBack, false>, grid, dim3(32), 0, s, p);
    return err == cudaSuccess ? launch_carry(p, s) : err;
}

template <class T>
cudaError_t back_t(const ScanParams &p, cudaStream_t s) {
    if (p.states <= 8) return back_w<T, 8, 1>(p, s);
    if (p.states <= 16) return back_w<T, 16, 1>(p, s);
    if (p.states <= 32) return back_w<T, 16, 2>(p, s);
    if (p.states <= 64) return back_w<T, 16, 4>(p, s);
    return back_w<T, 16, 8>(p, s);
}

}  // namespace

}  // namespace dwp
