// Gated delta rule, the states from chunk to chunk (and the outputs), and the
// walk back for the states' gradients.  A block has one sequence and head.
//
// Forward, a chunk:                          Back, from the last chunk:
//   P  = K S                                   X  = K dS,  Y = A^T dO
//   R  = beta (V - e^G P)                      dU = e^{G_C - G} X + scale Y
//   U  = T R                                   dR = T^T dU
//   S  = e^{G_C} S + K^T e^{G_C - G} U         dS = e^{G_C} dS + scale Q^T e^G dO - K^T beta e^G dR
//   O  = scale (e^G Q S + A U)
//
// All products are taken transposed, so that their 128 rows are the values
// and never a chunk's 64 rows: the state, f32 in registers (a thread has one
// value's row and half of the keys), goes to tensor memory as the first operand
// of the next products, as R and U do, and K, Q, T, A and dO are operands in
// shared memory as they are stored.  What is not itself bf16 is two bf16
// (split2), and of a product of two such the three larger parts are taken.
#pragma once

#include "delta.cuh"

namespace dwp {

namespace {

constexpr int kChainThreads = 256;
constexpr int kMostValues = 128;

// Shared memory of one chunk's inputs.
template <class T, int KD, bool kBack>
struct ChainStage {
    static constexpr int kP = kPieces<T>;
    static constexpr uint32_t kTileBytes = kChunk * kTileRow;  // of 64 x 64
    static constexpr uint32_t kKeys = kChunk * KD * 2, kValues = kChunk * kMostValues * 2;
    static constexpr int kWeightPieces = kBack || kP == 2 ? 2 : 1;
    static constexpr uint32_t k = 0, q = k + kP * kKeys, v = q + kP * kKeys;
    static constexpr uint32_t inverse = v + (kBack ? kP * kValues : kChunk * kMostValues * uint32_t(sizeof(T)));
    static constexpr uint32_t weights = inverse + 2 * kTileBytes, bytes = weights + kWeightPieces * kTileBytes;
    static constexpr int kStages = kP == 1 ? 2 : 1;
    static constexpr size_t kAll = 1024 + size_t(kStages) * bytes;
};

// Two planes of 64 x 64 as tiles.
template <int kCount>
__device__ __forceinline__ void load_planes(char *tile, const float *planes) {
    const char *src = reinterpret_cast<const char *>(planes);
#pragma unroll
    for (int e = threadIdx.x; e < kCount * kChunk * 8; e += kChainThreads) {
        const uint32_t plane = e / (kChunk * 8), r = e / 8 % kChunk, c = e % 8;
        copy16(smem_addr(tile + plane * kChunk * kTileRow + tile_piece(r, c)), src + size_t(e) * 16, 16u);
    }
}

template <class T, int KD, bool kBack, bool kWide>
__global__ void __launch_bounds__(kChainThreads, 1) delta_chain_kernel(DeltaBackwardParams bp) {
    using Stage = ChainStage<T, KD, kBack>;
    constexpr int kP = Stage::kP, kH = KD / 2;  // kH: keys of a thread
    extern __shared__ char raw[];
    __shared__ float beta_[2][kChunk], first_[2][kChunk], rest_[2][kChunk];
    __shared__ Sum2 sums[kChunk];
    __shared__ uint64_t bars[5];
    __shared__ uint32_t tmem;
    const DeltaParams &p = bp.f;
    char *sm = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
    const int half = warp / 4, dv = warp % 4 * 32 + lane, t0 = half * 32, k0 = half * kH;
    const int head = blockIdx.y, kh = head / (p.heads / p.key_heads), keys = p.keys, values = p.values;
    const int64_t seq = blockIdx.x;
    int64_t batch, row0, rows, slot0;
    delta_sequence(p, seq, batch, row0, rows, slot0);
    const int64_t chunks = (rows + kChunk - 1) / kChunk;
    const int kp = (keys + 7) / 8 * 8;

    if (tid == 0) {
        for (int i = 0; i < 5; ++i) mbar_init(&bars[i], 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem, 512);
    __syncthreads();
    // columns: sums of the first product; of the second; of the state's; then
    // operands: the state (hi, lo), R or U (hi, lo), U as it is or the queries' side (hi, lo)
    const uint32_t tm = tmem, mine = tm + (uint32_t(warp % 4) << 21);
    constexpr uint32_t kD0 = 0, kD1 = 64, kDS = 128, kS = 256, kR = 384, kU = 448;

    float S[kH];
    {
        const float *from = (kBack ? bp.grad_final : p.initial);
        const int64_t at = (seq * p.heads + head) * keys * values + dv;
#pragma unroll
        for (int k = 0; k < kH; ++k)
            S[k] = from && dv < values && k0 + k < keys ? from[at + int64_t(k0 + k) * values] : 0.0f;
    }
    auto chunk_of = [&](int64_t step) { return kBack ? chunks - 1 - step : step; };
    // a chunk's inputs to stage `st`; its decays and betas to registers of the last warp
    float g2[2], b2[2];
    auto load = [&](int64_t step, int st) {
        const int64_t c = chunk_of(step), row = row0 + c * kChunk, at = (slot0 + c) * p.heads + head;
        const int n = int(min(rows - c * kChunk, int64_t(kChunk)));
        char *s = sm + st * Stage::bytes;
        load_tile<T, kWide, kChunk, KD, kChainThreads>(s + Stage::k, Stage::kKeys, 0, p.k, batch, row, kh, n, keys);
        load_tile<T, kWide, kChunk, KD, kChainThreads>(s + Stage::q, Stage::kKeys, 0, p.q, batch, row, kh, n, keys);
        load_planes<2>(s + Stage::inverse, p.inverse + at * kChunk * kChunk);
        load_planes<Stage::kWeightPieces>(s + Stage::weights, p.weights + at * kChunk * kChunk);
        if constexpr (kBack) {
            load_tile<T, kWide, kChunk, kMostValues, kChainThreads>(s + Stage::v, Stage::kValues, 0, bp.grad_out, batch, row,
                                                                    head, n, values);
        } else {
            const T *src = delta_at<T>(p.v, batch, row, head);
            constexpr int kEach = 16 / int(sizeof(T)), kRow = kMostValues / kEach;
#pragma unroll
            for (int e = tid; e < kChunk * kRow; e += kChainThreads) {
                const int i = e / kRow, j = e % kRow * kEach, left = i < n ? values - j : 0;
                T *to = reinterpret_cast<T *>(s + Stage::v) + i * kMostValues + j;
                if constexpr (kWide) {
                    copy16(smem_addr(to), left > 0 ? src + int64_t(i) * p.v.row + j : src, left > 0 ? 16u : 0u);
                } else {
#pragma unroll
                    for (int l = 0; l < kEach; ++l) to[l] = l < left ? src[int64_t(i) * p.v.row + j + l] : from_f32<T>(0.0f);
                }
            }
        }
        if (warp == 7)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = lane + 32 * i;
                g2[i] = r < n ? delta_g(p.g, batch, row + r, head) : 0.0f;
                b2[i] = r < n ? delta_beta<T>(p, batch, row + r, head) : 0.0f;
            }
    };
    auto finish_load = [&](int st) {
        if (warp != 7) return;
        delta_sums(sums, [&](int i) { return i < 32 ? g2[0] : g2[1]; });
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = lane + 32 * i;
            const float e = __expf(sums[r].hi);
            beta_[st][r] = b2[i];
            first_[st][r] = fmaf(e, sums[r].lo, e);
            rest_[st][r] = __expf(sum2_less(sums[kChunk - 1], sums[r]));
        }
    };
    // the state as the next products' operand, and as kept for chunk `step`
    auto put_state = [&](int64_t step) {
        float *planes = kBack ? bp.ends : p.states;
        const bool keep = planes && step < chunks && dv < values;
        char *to = nullptr;
        if (keep)
            to = reinterpret_cast<char *>(planes + ((slot0 + chunk_of(step)) * p.heads + head) * kp * values) +
                 int64_t(dv) * kp * 2;
#pragma unroll
        for (int k = 0; k < kH; k += 16) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) split2(S[k + 2 * j], S[k + 2 * j + 1], hi[j], lo[j]);
            tmem_store<8>(mine + kS + (k0 + k) / 2, hi);
            tmem_store<8>(mine + kS + KD / 2 + (k0 + k) / 2, lo);
            if (keep)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (k0 + k + j * 8 < kp) {
                        char *at = to + (k0 + k + j * 8) * 2;
                        *reinterpret_cast<uint4 *>(at) = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
                        *reinterpret_cast<uint4 *>(at + int64_t(values) * kp * 2) =
                            make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
                    }
        }
        tmem_stored();
    };
    // 32 values of this thread's rows of the chunk, in two pieces, as an operand
    auto put_rows = [&](uint32_t at, const float (&x)[32]) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) split2(x[2 * j], x[2 * j + 1], hi[j], lo[j]);
        tmem_store<16>(mine + at + half * 16, hi);
        tmem_store<16>(mine + at + 32 + half * 16, lo);
    };
    auto meet = [&] {  // what was stored is there for the products
        tmem_stored();
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
    };
    bool ok = true;
    auto wait = [&](int bar, int64_t step) {
        if (ok) ok = mma_wait(&bars[bar], uint32_t(step & 1));
        tmem_fence_after();
    };
    auto read = [&](float (&x)[32], uint32_t at) {
        uint32_t v[32];
        tmem_load<32>(v, mine + at);
        tmem_ready();
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]);
    };

    if (chunks > 0) {
        load(0, 0);
        put_state(0);
        finish_load(0);
    }
    float o1[32];  // forward: what the state gives to the outputs
    // forward: the outputs of chunk `step`
    auto put_out = [&](int64_t step) {
        const int64_t c = step, row = row0 + c * kChunk;
        const int n = int(min(rows - c * kChunk, int64_t(kChunk)));
        float o2[32];
        read(o2, kD1 + t0);
        if (dv >= values) return;
        T *out = delta_at<T>(p.out, batch, row + t0, head) + dv;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (t0 + j < n) out[int64_t(j) * p.out.row] = from_f32<T>(ok ? fmaf(p.scale, o2[j], o1[j]) : __int_as_float(0x7fffffff));
    };
    for (int64_t step = 0; step < chunks; ++step) {
        const int st = Stage::kStages == 2 ? int(step & 1) : 0, vs = int(step & 1);
        const int64_t at = (slot0 + chunk_of(step)) * p.heads + head;
        char *s = sm + st * Stage::bytes;
        copies_done();
        fence_proxy_async_smem();
        meet();
        const Operand<kChunk, false> K(s + Stage::k), Kl(s + Stage::k + Stage::kKeys);
        const Operand<kChunk, true> Ko(s + Stage::k), Klo(s + Stage::k + Stage::kKeys);
        if (warp == 0 && elect_one()) {
            product_ts<kChunk, KD>(tm + kD0, tm + kS, K, false);
            product_ts<kChunk, KD>(tm + kD0, tm + kS + KD / 2, K, true);
            if constexpr (kP == 2) product_ts<kChunk, KD>(tm + kD0, tm + kS, Kl, true);
            mma_commit(&bars[0]);
            if constexpr (kBack) {
                const Operand<kChunk, true> dO(s + Stage::v), dOl(s + Stage::v + Stage::kValues), A(s + Stage::weights),
                    Al(s + Stage::weights + Stage::kTileBytes);
                product_ss<kChunk, kChunk>(tm + kD1, dO, A, false);
                product_ss<kChunk, kChunk>(tm + kD1, dO, Al, true);
                if constexpr (kP == 2) product_ss<kChunk, kChunk>(tm + kD1, dOl, A, true);
            } else {
                const Operand<kChunk, false> Q(s + Stage::q), Ql(s + Stage::q + Stage::kKeys);
                product_ts<kChunk, KD>(tm + kDS, tm + kS, Q, false);
                if constexpr (kP == 2) {
                    product_ts<kChunk, KD>(tm + kDS, tm + kS + KD / 2, Q, true);
                    product_ts<kChunk, KD>(tm + kDS, tm + kS, Ql, true);
                }
            }
            mma_commit(&bars[1]);
        }
        // the last products that read the other stage have ended
        if (!kBack && step > 0) wait(4, step - 1);
        if (Stage::kStages == 2 && step + 1 < chunks) load(step + 1, st ^ 1);
        const float *beta = beta_[vs], *first = first_[vs], *rest = rest_[vs];
        const float whole = first[kChunk - 1];
        float x[32], y[32];
        if constexpr (!kBack) {
            if (step > 0) put_out(step - 1);
            wait(0, step);
            read(x, kD0 + t0);
            const T *v = reinterpret_cast<const T *>(s + Stage::v) + t0 * kMostValues + dv;
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = beta[t0 + j] * fmaf(-first[t0 + j], x[j], to_f32<T>(v[j * kMostValues]));
            put_rows(kR, x);
            wait(1, step);
            read(o1, kDS + t0);
#pragma unroll
            for (int j = 0; j < 32; ++j) o1[j] *= p.scale * first[t0 + j];
        } else {
            // the queries' side: scale e^G dO
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const uint32_t e = tile_at(t0 + j, dv, kChunk);
                float f = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(s + Stage::v + e));
                if constexpr (kP == 2)
                    f += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(s + Stage::v + Stage::kValues + e));
                x[j] = p.scale * first[t0 + j] * f;
            }
            put_rows(kU, x);
            wait(0, step);
            read(x, kD0 + t0);
            wait(1, step);
            read(y, kD1 + t0);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = fmaf(rest[t0 + j], x[j], p.scale * y[j]);
            put_rows(kR, x);
        }
        meet();
        if (warp == 0 && elect_one()) {
            const Operand<kChunk, kBack> inv(s + Stage::inverse), invl(s + Stage::inverse + Stage::kTileBytes);
            product_ts<kChunk, kChunk>(tm + kD0, tm + kR, inv, false);
            product_ts<kChunk, kChunk>(tm + kD0, tm + kR + 32, inv, true);
            product_ts<kChunk, kChunk>(tm + kD0, tm + kR, invl, true);
            mma_commit(&bars[2]);
        }
        wait(2, step);
        read(x, kD0 + t0);
        if (float *keep = kBack ? bp.dr : p.u; keep && dv < values) {
            keep += at * kChunk * values + int64_t(t0) * values + dv;
#pragma unroll
            for (int j = 0; j < 32; ++j) keep[j * values] = x[j];
        }
        if constexpr (!kBack) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if constexpr (kP == 2) split2(x[2 * j], x[2 * j + 1], hi[j], lo[j]);
                else hi[j] = round2(x[2 * j], x[2 * j + 1]);
            }
            tmem_store<16>(mine + kU + half * 16, hi);
            if constexpr (kP == 2) tmem_store<16>(mine + kU + 32 + half * 16, lo);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] *= kBack ? -beta[t0 + j] * first[t0 + j] : rest[t0 + j];
        put_rows(kR, x);
        meet();
        if (warp == 0 && elect_one()) {
            product_ts<KD, kChunk>(tm + kDS, tm + kR, Ko, false);
            product_ts<KD, kChunk>(tm + kDS, tm + kR + 32, Ko, true);
            if constexpr (kP == 2) product_ts<KD, kChunk>(tm + kDS, tm + kR, Klo, true);
            if constexpr (kBack) {
                const Operand<kChunk, true> Q(s + Stage::q), Ql(s + Stage::q + Stage::kKeys);
                product_ts<KD, kChunk>(tm + kDS, tm + kU, Q, true);
                product_ts<KD, kChunk>(tm + kDS, tm + kU + 32, Q, true);
                if constexpr (kP == 2) product_ts<KD, kChunk>(tm + kDS, tm + kU, Ql, true);
            }
            mma_commit(&bars[3]);
            if constexpr (!kBack) {
                const Operand<kChunk, false> A(s + Stage::weights), Al(s + Stage::weights + Stage::kTileBytes);
                product_ts<kChunk, kChunk>(tm + kD1, tm + kU, A, false);
                if constexpr (kP == 2) {
                    product_ts<kChunk, kChunk>(tm + kD1, tm + kU + 32, A, true);
                    product_ts<kChunk, kChunk>(tm + kD1, tm + kU, Al, true);
                }
                mma_commit(&bars[4]);
            }
        }
        wait(3, step);
#pragma unroll
        for (int k = 0; k < kH; k += 32) {
            read(x, kDS + k0 + k);
#pragma unroll
            for (int j = 0; j < 32; ++j) S[k + j] = fmaf(whole, S[k + j], x[j]);
        }
        if (step + 1 < chunks) {
            if (Stage::kStages == 1) {
                // the last products and reads of this stage end first
                if constexpr (!kBack) wait(4, step);
                __syncthreads();
                load(step + 1, 0);
            }
            put_state(step + 1);
            finish_load(vs ^ 1);
        }
    }
    if constexpr (!kBack)
        if (chunks > 0) {
            wait(4, chunks - 1);
            put_out(chunks - 1);
        }
    if (float *to = kBack ? bp.grad_initial : p.final; to && dv < values) {
        to += (seq * p.heads + head) * keys * values + dv;
#pragma unroll
        for (int k = 0; k < kH; ++k)
            if (k0 + k < keys) to[int64_t(k0 + k) * values] = ok ? S[k] : __int_as_float(0x7fffffff);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 0) tmem_free(tm, 512);
}

template <class T, int KD, bool kBack, bool kWide>
cudaError_t chain_k(const DeltaBackwardParams &p, cudaStream_t s) {
    const auto kernel = delta_chain_kernel<T, KD, kBack, kWide>;
    constexpr size_t bytes = ChainStage<T, KD, kBack>::kAll;
    if (device_blocks(reinterpret_cast<const void *>(kernel), kChainThreads, bytes) == 0) return cudaErrorInvalidConfiguration;
    return launch_pdl(kernel, dim3(uint32_t(p.f.sequences), uint32_t(p.f.heads)), dim3(kChainThreads), bytes, s, p);
}

template <class T, bool kBack>
cudaError_t chain_t(const DeltaBackwardParams &p, cudaStream_t s) {
    if (p.f.keys <= 64) return p.f.wide ? chain_k<T, 64, kBack, true>(p, s) : chain_k<T, 64, kBack, false>(p, s);
    return p.f.wide ? chain_k<T, 128, kBack, true>(p, s) : chain_k<T, 128, kBack, false>(p, s);
}

}  // namespace

}  // namespace dwp
