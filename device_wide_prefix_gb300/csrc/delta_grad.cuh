// Gated delta rule, the gradients of a chunk's rows, from the state before it,
// its corrections U, the gradient of the state after it and that of the
// corrections' right sides, dR:
//
//   dA = scale exp(G_i - G_j) dO_i.U_j (j <= i),  E = -exp(G_i - G_j) dR_i.U_j (j < i)
//   dQ = scale e^G dO S0^T + dA K
//   Z  = E K - e^G dR S0^T,   Y = e^{G_C - G} U dS1^T + dA^T Q + (beta E)^T K
//   dK = beta Z + Y,   dV = beta dR,   dbeta = dR.V + k.Z
//   dG = q.dQ + beta k.Z - k.Y, and <S1, dS1> at the chunk's last row; dg its
//   sum from the last row down
//
// (dG: G_i is in e^{G_i} q_i and, as e^{G_i} beta_i k_i and e^{-G_i} k_i, in
// what k_i does first and what it does to later rows.)
//
// A block has one chunk and key head and goes over the heads that share it,
// adding their dQ and dK in registers.  The products with the states and the
// second ones have the keys as rows and the chunk's rows as columns; dA and E
// come from one product of [dO; dR] with U.  Numbers that are not bf16 are in
// two pieces, as in the chain.
#pragma once

#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kGradThreads = 256;
constexpr int kMost = 128;  // keys and values, zeros past their own count

template <class T>
struct GradSpace {
    static constexpr int kP = kPieces<T>;
    static constexpr uint32_t kRows = kChunk * kMost * 2, kState = kMost * kMost * 2;
    // keys and queries; [dO; dR] (hi, lo), later [dA; E] and beta E; U (hi, lo);
    // the state before the chunk, later the gradient of the one after it (hi, lo)
    static constexpr uint32_t k = 0, q = k + kP * kRows, stack = q + kP * kRows, u = stack + 4 * kRows;
    static constexpr uint32_t state = u + 2 * kRows, bytes = state + 2 * kState;
    static constexpr uint32_t cross = stack, scaled = stack + 2 * kRows;
    static constexpr size_t kAll = 1024 + bytes;
};

// Sums over the 32 lanes of each of 32 numbers: lane l gets that of number l.
__device__ __forceinline__ float sums_of_32(float (&x)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float give = up ? x[j] : x[j + o], keep = up ? x[j + o] : x[j];
            x[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    return x[0];
}

// 64 rows of f32, `dim` columns, to a tile in two pieces from row `first` on.
template <class F>
__device__ __forceinline__ void load_f32_rows(char *hi, char *lo, uint32_t tile_rows, int first, const float *src, int dim,
                                              bool wide, F each) {
    for (int e = threadIdx.x; e < kChunk * kMost / 8; e += kGradThreads) {
        const int i = e / (kMost / 8), c = e % (kMost / 8), left = dim - c * 8;
        const uint32_t at = uint32_t(c / 8) * tile_rows * kTileRow + tile_piece(uint32_t(first + i), uint32_t(c % 8));
        float f[8];
        if (wide) load_eight<float, true>(f, src + int64_t(i) * dim + c * 8, left);
        else load_eight<float, false>(f, src + int64_t(i) * dim + c * 8, left);
        store_pieces(hi, lo, at, f);
        each(i, c * 8, left, f);
    }
}

__device__ __forceinline__ float2 pair_of(uint32_t hi, uint32_t lo) {
    return make_float2(__uint_as_float(hi << 16) + __uint_as_float(lo << 16),
                       __uint_as_float(hi & 0xffff0000u) + __uint_as_float(lo & 0xffff0000u));
}

template <class T, bool kWide>
__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(DeltaBackwardParams bp) {
    using Space = GradSpace<T>;
    constexpr int kP = Space::kP;
    constexpr uint32_t kRows = Space::kRows, kState = Space::kState;
    extern __shared__ char raw[];
    __shared__ Sum2 sums[kChunk];
    __shared__ float beta[kChunk], first[kChunk], rest[kChunk], value_dot[kChunk];
    __shared__ uint64_t bars[4];
    __shared__ uint32_t tmem;
    const DeltaParams &p = bp.f;
    char *sm = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
    // sums over the keys, in U's place when its products have ended
    struct Dots {
        float key[4][kChunk], all[4][kChunk], whole[kGradThreads / 32];
    };
    Dots &dots = *reinterpret_cast<Dots *>(sm + Space::u);
    pdl_trigger();
    pdl_wait();
    const DeltaChunk c = delta_chunk(p, blockIdx.x);
    if (c.rows == 0) return;
    const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
    const int half = warp / 4, dk = warp % 4 * 32 + lane, t0 = half * 32, n = c.rows;
    const int kh = blockIdx.y, per = p.heads / p.key_heads, keys = p.keys, values = p.values, tiles = (keys + 63) / 64;
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&bars[i], 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem, 512);
    load_tile<T, kWide, kChunk, kMost, kGradThreads>(tid, sm + Space::k, kRows, 0, p.k, c.batch, c.row, kh, n, keys);
    load_tile<T, kWide, kChunk, kMost, kGradThreads>(tid, sm + Space::q, kRows, 0, p.q, c.batch, c.row, kh, n, keys);
    // of the states' tiles what no state fills
    for (int e = tid; e < 2 * kMost * kMost / 8; e += kGradThreads)
        if (e / 8 % kMost >= values || e / (kMost * 8) % 2 >= tiles)
            *reinterpret_cast<uint4 *>(sm + Space::state + uint32_t(e) * 16) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const uint32_t tm = tmem, mine = tm + (uint32_t(warp % 4) << 21);
    constexpr uint32_t kDX = 0, kDA = 128, kDW = 192, kDY = 320, kDU = 384;
    bool ok = true;
    auto read = [&](float (&x)[32], uint32_t at) {
        uint32_t v[32];
        tmem_load<32>(v, mine + at);
        tmem_ready();
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]);
    };
    auto meet = [&] {
        copies_done();
        fence_proxy_async_smem();
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
    };
    // a key's or query's entry `dk` of row i
    auto entry = [&](uint32_t tile, int i) {
        const char *at = sm + tile + tile_at(uint32_t(i), uint32_t(dk), kChunk);
        float f = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(at));
        if constexpr (kP == 2) f += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(at + kRows));
        return f;
    };
    float dq[32], dkey[32];
    for (int h = 0; h < per; ++h) {
        const int head = kh * per + h;
        const int64_t at = int64_t(blockIdx.x) * p.heads + head;
        const uint32_t parity = uint32_t(h & 1);
        auto wait = [&](int bar) {
            if (ok) ok = mma_wait(&bars[bar], parity);
            tmem_fence_after();
        };
        // the state before the chunk, as it was kept
        const char *S0 = reinterpret_cast<const char *>(p.states + at * tiles * 64 * values);
        const char *S1 = reinterpret_cast<const char *>(bp.ends + at * tiles * 64 * values);
        if (tid == 0) {
            const uint32_t each = uint32_t(values) * kTileRow;
            mbar_arrive_expect_tx(&bars[3], 2 * tiles * each);
            for (int i = 0; i < 2 * tiles; ++i)
                bulk_load(sm + Space::state + i / tiles * kState + i % tiles * kMost * kTileRow, S0 + int64_t(i) * each, each,
                          &bars[3]);
        }
        load_tile<T, kWide, 2 * kChunk, kMost, kGradThreads>(tid, sm + Space::stack, 2 * kRows, 0, bp.grad_out, c.batch, c.row,
                                                             head, n, values);
        if constexpr (kP == 1)  // its second piece
            for (int e = tid; e < kChunk * kMost / 8; e += kGradThreads) {
                const uint32_t i = e / (kMost / 8), j = e % (kMost / 8);
                *reinterpret_cast<uint4 *>(sm + Space::stack + 2 * kRows + j / 8 * 2 * kChunk * kTileRow +
                                           tile_piece(i, j % 8)) = make_uint4(0, 0, 0, 0);
            }
        if (warp == 7) {
            float g[2];
            Sum2 s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane + 32 * i;
                g[i] = r < n ? delta_g(p.g, c.batch, c.row + r, head) : 0.0f;
                beta[r] = r < n ? delta_beta<T>(p, c.batch, c.row + r, head) : 0.0f;
            }
            delta_sums(s, g);
            const Sum2 last = {__shfl_sync(0xffffffffu, s[1].hi, 31), __shfl_sync(0xffffffffu, s[1].lo, 31)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float e = __expf(s[i].hi);
                sums[lane + 32 * i] = s[i];
                first[lane + 32 * i] = fmaf(e, s[i].lo, e);
                rest[lane + 32 * i] = __expf(sum2_less(last, s[i]));
            }
        }
        __syncthreads();
        const bool wide_values = values % 4 == 0;
        load_f32_rows(sm + Space::stack, sm + Space::stack + 2 * kRows, 2 * kChunk, kChunk, bp.dr + at * kChunk * values, values,
                      wide_values, [&](int i, int j0, int left, const float (&f)[8]) {
                          // the row's share of dR.V, and dV
                          float s = 0.0f;
                          if (i < n && left > 0) {
                              float v[8], d[8];
                              load_eight<T, kWide>(v, delta_at<T>(p.v, c.batch, c.row + i, head) + j0, left);
                              T *to = delta_at<T>(bp.grad_v, c.batch, c.row + i, head) + j0;
#pragma unroll
                              for (int j = 0; j < 8; ++j) s = fmaf(f[j], v[j], s), d[j] = beta[i] * f[j];
                              // dense rows of whole 16-byte pieces start on 16 bytes if the first does
                              if (kWide && bp.wide && left >= 8) {
                                  store_f32<8>(to, d);
                              } else {
#pragma unroll
                                  for (int j = 0; j < 8; ++j)
                                      if (j < left) to[j] = from_f32<T>(d[j]);
                              }
                          }
#pragma unroll
                          for (int o = 8; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
                          if (lane % 16 == 0) value_dot[i] = s;
                      });
        load_f32_rows(sm + Space::u, sm + Space::u + kRows, kChunk, 0, p.u + at * kChunk * values, values, wide_values,
                      [](int, int, int, const float (&)[8]) {});
        if (ok) ok = mma_wait(&bars[3], parity);
        meet();
        const Operand<kChunk, false> U(sm + Space::u), Ul(sm + Space::u + kRows);
        const Operand<kMost, true> S(sm + Space::state), Sl(sm + Space::state + kState);
        if (warp == 0 && elect_one()) {
            const Operand<2 * kChunk, false> both(sm + Space::stack), bothl(sm + Space::stack + 2 * kRows);
            product_ss<kChunk, kMost>(tm + kDA, both, U, false);
            product_ss<kChunk, kMost>(tm + kDA, both, Ul, true);
            product_ss<kChunk, kMost>(tm + kDA, bothl, U, true);
            mma_commit(&bars[0]);
            product_ss<2 * kChunk, kMost>(tm + kDX, S, both, false);
            product_ss<2 * kChunk, kMost>(tm + kDX, Sl, both, true);
            if constexpr (kP == 2) {
                product_ss<2 * kChunk, kMost>(tm + kDX, S, bothl, true);
            } else {
                const Operand<2 * kChunk, false> drl(sm + Space::stack + 2 * kRows + kChunk * kTileRow);
                product_ss<kChunk, kMost>(tm + kDX + kChunk, S, drl, true);
            }
            mma_commit(&bars[1]);
        }
        // dA and E, this thread's row and half of the columns
        float w[32];
        wait(0);
        read(w, kDA + t0);
        const int row = dk % kChunk;
        const bool cross = dk >= kChunk;
        {
            const Sum2 own = sums[row];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const int col = t0 + j;
                const bool in = cross ? col < row : col <= row;
                w[j] = in ? (cross ? -1.0f : p.scale) * __expf(sum2_less(own, sums[col])) * w[j] : 0.0f;
            }
        }
        wait(1);
        __syncthreads();  // every thread's products from the stack have ended, and their reads of it
        {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[8];
#pragma unroll
                for (int l = 0; l < 8; ++l) f[l] = w[j * 8 + l];
                store_pieces(sm + Space::cross, sm + Space::cross + kRows, tile_piece(uint32_t(dk), uint32_t(half * 4 + j)), f);
                if (cross) {
#pragma unroll
                    for (int l = 0; l < 8; ++l) f[l] *= beta[row];
                    store_pieces(sm + Space::scaled, sm + Space::scaled + kChunk * kTileRow,
                                 tile_piece(uint32_t(row), uint32_t(half * 4 + j)), f);
                }
            }
        }
        // the gradient of the state after the chunk takes the state's place, and meets it on the way
        float meeting = 0.0f;
#pragma unroll 4
        for (int e = tid; e < tiles * values * 8; e += kGradThreads) {
            const uint4 hi = *reinterpret_cast<const uint4 *>(S1 + e * 16);
            const uint4 lo = *reinterpret_cast<const uint4 *>(S1 + (tiles * values * 8 + e) * 16);
            uint4 *at_hi = reinterpret_cast<uint4 *>(sm + Space::state + (e >= values * 8 ? kMost * 8 + e - values * 8 : e) * 16);
            uint4 *at_lo = reinterpret_cast<uint4 *>(reinterpret_cast<char *>(at_hi) + kState);
            const uint4 shi = *at_hi, slo = *at_lo;
            auto with = [&](uint32_t a, uint32_t b, uint32_t x, uint32_t y) {
                const float2 f = pair_of(a, b), g = pair_of(x, y);
                meeting = fmaf(f.x, g.x, fmaf(f.y, g.y, meeting));
            };
            with(hi.x, lo.x, shi.x, slo.x), with(hi.y, lo.y, shi.y, slo.y);
            with(hi.z, lo.z, shi.z, slo.z), with(hi.w, lo.w, shi.w, slo.w);
            *at_hi = hi, *at_lo = lo;
        }
        meeting *= first[kChunk - 1];
        meet();
        if (warp == 0 && elect_one()) {
            const Operand<kChunk, true> K(sm + Space::k), Q(sm + Space::q);
            const Operand<2 * kChunk, false> W(sm + Space::cross), Wl(sm + Space::cross + kRows);
            const Operand<2 * kChunk, true> A(sm + Space::cross), Al(sm + Space::cross + kRows);
            const Operand<kChunk, true> E(sm + Space::scaled), El(sm + Space::scaled + kChunk * kTileRow);
            product_ss<2 * kChunk, kChunk>(tm + kDW, K, W, false);
            product_ss<2 * kChunk, kChunk>(tm + kDW, K, Wl, true);
            product_ss<kChunk, kChunk>(tm + kDY, Q, A, false);
            product_ss<kChunk, kChunk>(tm + kDY, Q, Al, true);
            product_ss<kChunk, kChunk>(tm + kDY, K, E, true);
            product_ss<kChunk, kChunk>(tm + kDY, K, El, true);
            if constexpr (kP == 2) {
                const Operand<kChunk, true> Kl(sm + Space::k + kRows), Ql(sm + Space::q + kRows);
                product_ss<2 * kChunk, kChunk>(tm + kDW, Kl, W, true);
                product_ss<kChunk, kChunk>(tm + kDY, Ql, A, true);
                product_ss<kChunk, kChunk>(tm + kDY, Kl, E, true);
            }
            product_ss<kChunk, kMost>(tm + kDU, S, U, false);
            product_ss<kChunk, kMost>(tm + kDU, S, Ul, true);
            product_ss<kChunk, kMost>(tm + kDU, Sl, U, true);
            mma_commit(&bars[2]);
        }
        wait(2);
        float x[32], key_sum[32], all_sum[32];
        // dQ
        read(w, kDX + t0);
        read(x, kDW + t0);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float d = fmaf(p.scale * first[t0 + j], w[j], x[j]);
            dq[j] = h ? dq[j] + d : d;
            all_sum[j] = d * entry(Space::q, t0 + j);
        }
        // Z
        read(w, kDX + kChunk + t0);
        read(x, kDW + kChunk + t0);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float z = fmaf(-first[t0 + j], w[j], x[j]), b = beta[t0 + j] * z, k = entry(Space::k, t0 + j);
            dkey[j] = h ? dkey[j] + b : b;
            key_sum[j] = k * z;
            all_sum[j] = fmaf(k, b, all_sum[j]);
        }
        // Y
        read(w, kDU + t0);
        read(x, kDY + t0);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float r = rest[t0 + j] * w[j], y = r + x[j], k = entry(Space::k, t0 + j);
            meeting = fmaf(k, r, meeting);
            dkey[j] += y;
            all_sum[j] = fmaf(-k, y, all_sum[j]);
        }
        const float a = sums_of_32(all_sum, lane), b = sums_of_32(key_sum, lane);
        dots.all[warp % 4][t0 + lane] = a, dots.key[warp % 4][t0 + lane] = b;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) meeting += __shfl_xor_sync(0xffffffffu, meeting, o);
        if (lane == 0) dots.whole[warp] = meeting;
        tmem_fence_before();
        __syncthreads();
        if (warp == 7) {
            float whole = 0.0f;
            for (int w = 0; w < kGradThreads / 32; ++w) whole += dots.whole[w];
            const float bad = ok ? 0.0f : __int_as_float(0x7fffffff);
            float g[2];
            Sum2 sum[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = kChunk - 1 - (lane + 32 * r);
                g[r] = i >= n ? 0.0f : (dots.all[0][i] + dots.all[1][i]) + (dots.all[2][i] + dots.all[3][i]) +
                                           (i == n - 1 ? whole : 0.0f) + bad;
            }
            delta_sums(sum, g);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = kChunk - 1 - (lane + 32 * r);
                if (i >= n) continue;
                if (bp.grad_g.data) *delta_at<float>(bp.grad_g, c.batch, c.row + i, head) = sum[r].hi;
                const float d = value_dot[i] + ((dots.key[0][i] + dots.key[1][i]) + (dots.key[2][i] + dots.key[3][i])) + bad;
                if (p.beta_f32) *delta_at<float>(bp.grad_beta, c.batch, c.row + i, head) = d;
                else *delta_at<T>(bp.grad_beta, c.batch, c.row + i, head) = from_f32<T>(d);
            }
        }
    }
    if (dk < keys) {
        T *to_q = delta_at<T>(bp.grad_q, c.batch, c.row + t0, kh) + dk, *to_k = delta_at<T>(bp.grad_k, c.batch, c.row + t0, kh) + dk;
        const float bad = ok ? 0.0f : __int_as_float(0x7fffffff);
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (t0 + j < n) {
                to_q[j * bp.grad_q.row] = from_f32<T>(dq[j] + bad);
                to_k[j * bp.grad_k.row] = from_f32<T>(dkey[j] + bad);
            }
    }
    __syncthreads();
    if (warp == 0) tmem_free(tm, 512);
}

template <class T, bool kWide>
cudaError_t grad_k(const DeltaBackwardParams &p, cudaStream_t s) {
    const auto kernel = delta_grad_kernel<T, kWide>;
    constexpr size_t bytes = GradSpace<T>::kAll;
    if (device_blocks(reinterpret_cast<const void *>(kernel), kGradThreads, bytes) == 0) return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, dim3(uint32_t(p.f.slots), uint32_t(p.f.key_heads)), dim3(kGradThreads), bytes, s, p);
}

template <class T>
cudaError_t grad_t(const DeltaBackwardParams &p, cudaStream_t s) {
    return p.f.wide ? grad_k<T, true>(p, s) : grad_k<T, false>(p, s);
}

}  // namespace

}  // namespace dwp
