// Gradient of the selective state space scan.  With dy = dout * silu(z), per
// channel d and state n, rows from last to first:
//
//   dh[t] = C[t,n] dy[t] + a[t+1] dh[t+1]        (a = exp(delta A))
//   dC[t,n] = sum_d dy h[t],   dB[t,n] = sum_d dh delta u
//   q1 = sum_n dh B,           q2 = sum_n dh a h[t-1] A
//   du = delta q1 + D dy,      ddelta = u q1 + q2
//   dA = sum_t dh a h[t-1] delta
//
// A block is one warp that walks its channels backward through its rows, a
// tile of kCheckpointRows at a time.  The states come again from the one the
// forward kept before the tile: a first walk leaves the states before every
// kSub rows in shared memory; then, from the last kSub rows to the first, a
// second walk forward keeps the states before each row in registers, and the
// walk backward uses them.
//
// NL neighbouring lanes share a pair of channels, each with NT states of
// both.  A sum over states (q1, q2, y) takes one exchange between the two
// lanes of a pair plus log2(NL) - 1 more; a sum over channels (dB, dC) goes
// over the 32 / NL pairs by halves, each exchange halving the values a lane
// still holds.  The states' order within a lane depends on the lane's pair
// (which of its state pairs comes first), so that the half to keep is in the
// same registers in every lane and no value has to be selected.
#pragma once

#include "selscan.cuh"

namespace dwp {

namespace {

constexpr int kSub = 4;
constexpr int kSubs = kCheckpointRows / kSub;
constexpr int kTile = kCheckpointRows;

template <class T, int NT, int NL>
__global__ void __launch_bounds__(32, 8) selscan_backward_kernel(ScanBackwardParams q) {
    constexpr int kC = 64 / NL, kN = NT * NL, kP = NT / 2;
    const ScanParams &p = q.f;
    __shared__ float2 sd[kTile * kC];                   // (delta, delta u)
    __shared__ float sg[kTile * kC];                    // dy
    __shared__ float s1[kTile * kC], s2[kTile * kC], sy[kTile * kC];
    __shared__ float2 sbc[kTile * kN];                  // B, then C, of each row
    __shared__ float2 sh[(kSubs - 1) * 2 * kP * 32];    // states before rows kSub, 2 kSub, ...
    pdl_trigger();
    pdl_wait();

    const int lane = threadIdx.x, nl = lane % NL, n0 = nl * NT, pair = lane / NL;
    const uint32_t b = blockIdx.x / uint32_t(p.chunks), chunk = blockIdx.x % uint32_t(p.chunks);
    const int64_t t0 = int64_t(chunk) * p.chunk_rows;
    const int64_t t1 = min(t0 + p.chunk_rows, p.rows);
    const uint32_t g = blockIdx.y / p.group_blocks, gb = blockIdx.y % p.group_blocks;
    const int64_t cg = int64_t(gb) * kC;
    const int64_t cb = int64_t(g) * p.group + cg;
    const int live = int(min(int64_t(kC), p.group - cg));
    const int own = pair * 2 + (lane & 1), other = own ^ 1;
    // state pair j of this lane is pair j ^ flip of its NT states
    const int flip = kP == 4 ? (pair & 1) * 2 + (pair >> 1 & 1) : pair & 1;

    F2 A2[2][kP], e[2][kP], dA[2][kP], h[2][kP];
    const F2 zero = f2(0.0f, 0.0f);
    const bool whole = p.states == kN && p.states_wide;  // every state is live, in aligned pairs
    auto load_state = [&](F2(&v)[2][kP], const float *from, int64_t i) {
        if (!from) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < kP; ++j) v[c][j] = zero;
            return;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // a channel past the last takes the last's
            const float *x = from + (i * p.channels + cb + min(c ? other : own, live - 1)) * p.states + n0;
            if (whole) {
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const float2 s = *reinterpret_cast<const float2 *>(x + 2 * (j ^ flip));
                    v[c][j] = f2(s.x, s.y);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const int n = 2 * (j ^ flip);
                    v[c][j] = f2(n0 + n < p.states ? x[n] : 0.0f, n0 + n + 1 < p.states ? x[n + 1] : 0.0f);
                }
            }
        }
    };
    auto save_state = [&](float *to, int64_t i, const F2(&v)[2][kP]) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                const int n = n0 + 2 * (j ^ flip), ch = c ? other : own;
                float *x = to + (i * p.channels + cb + ch) * p.states + n;
                const float2 s = unpack(v[c][j]);
                if (ch < live && n < p.states) x[0] = s.x;
                if (ch < live && n + 1 < p.states) x[1] = s.y;
            }
    };
    load_state(A2, p.A, 0);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < kP; ++j) A2[c][j] = decay_rate(A2[c][j]);
    // the walk back's entry k is the state after it left the last chunk but k
    if (chunk + 1 < p.chunks) load_state(e, p.carry, int64_t(b) * (p.chunks - 1) + (p.chunks - 2 - chunk));
    else load_state(e, p.segmap ? nullptr : q.grad_final, b);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < kP; ++j) dA[c][j] = zero;

    const T *u = static_cast<const T *>(p.u) + int64_t(b) * p.u_batch + cb;
    const T *dt = static_cast<const T *>(p.dt) + int64_t(b) * p.dt_batch + cb;
    const T *z = p.z ? static_cast<const T *>(p.z) + int64_t(b) * p.z_batch + cb : u;
    const int64_t z_row = p.z ? p.z_row : p.u_row;
    const T *B = static_cast<const T *>(p.B) + int64_t(b) * p.b_batch + g * p.b_group;
    const T *C = static_cast<const T *>(p.C) + int64_t(b) * p.c_batch + g * p.c_group;
    const T *go = static_cast<const T *>(q.grad_out) + int64_t(b) * q.grad_batch + cb;
    // gradients of the inputs are dense
    const int64_t out0 = int64_t(b) * p.rows * p.channels + cb;
    T *gu = static_cast<T *>(q.grad_u) + out0, *gdt = static_cast<T *>(q.grad_dt) + out0;
    T *gz = p.z ? static_cast<T *>(q.grad_z) + out0 : nullptr;

    // per channel work: channel `mine`, rows from `mine_row` on by kMineRows
    constexpr int kMineRows = 32 / kC, kMine = kTile / kMineRows;
    const int mine = lane % kC, mine_row = lane / kC;
    const uint32_t mine_at = uint32_t(min(mine, live - 1));
    const float bias = p.dt_bias ? p.dt_bias[cb + mine_at] : 0.0f, Dv = p.D ? p.D[cb + mine_at] : 0.0f;
    float acc_D = 0.0f, acc_bias = 0.0f;

    // where this lane's share of dB or dC ends up: see reduce()
    float *bc_out = q.partial_bc + ((int64_t(gb) * p.batch + b) * p.rows * p.groups + g) * 2 * p.states;
    const int64_t bc_row = p.groups * 2 * p.states;

    auto tile = [&](int64_t s0, int rows, uint32_t code, auto look) {
        constexpr bool kLook = decltype(look)::value;
        auto flag = [&](int r) -> uint32_t { return kLook ? __shfl_sync(0xffffffffu, code, r) : 0u; };
        load_state(h, p.checkpoints, int64_t(b) * p.tiles + s0 / kTile);
        // the step past row r; y: this lane's part of C h
        auto step = [&](int r, bool with_y, float (&y)[2]) {
            const float2 d0 = sd[r * kC + own], d1 = sd[r * kC + other];
            const F2 dd[2] = {f2(d0.x, d0.x), f2(d1.x, d1.x)}, xx[2] = {f2(d0.y, d0.y), f2(d1.y, d1.y)};
            F2 acc[2] = {zero, zero};
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                const float2 bv = sbc[r * kN + (n0 / 2 + (j ^ flip))];
                float2 cv;
                if (with_y) cv = sbc[r * kN + kN / 2 + (n0 / 2 + (j ^ flip))];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float2 ar = unpack(mul2(dd[c], A2[c][j]));
                    h[c][j] = fma2(f2(ex2(ar.x), ex2(ar.y)), h[c][j], mul2(xx[c], f2(bv.x, bv.y)));
                    if (with_y) acc[c] = fma2(f2(cv.x, cv.y), h[c][j], acc[c]);
                }
            }
            if (with_y) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float2 s = unpack(acc[c]);
                    y[c] = s.x + s.y;
                }
            }
        };
        float none[2];
#pragma unroll 1
        for (int k = 0; k + 1 < kSubs; ++k) {
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const uint32_t f = flag(k * kSub + i);
                if (kLook && f == kRowOutside) continue;
                if (kLook && (f & kRowHead)) load_state(h, p.initial, f & kRowSegment);
                step(k * kSub + i, false, none);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < kP; ++j) sh[((k * 2 + c) * kP + j) * 32 + lane] = unpack(h[c][j]);
        }
#pragma unroll 1
        for (int k = kSubs - 1; k >= 0; --k) {
            if (k == 0) {
                load_state(h, p.checkpoints, int64_t(b) * p.tiles + s0 / kTile);
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int j = 0; j < kP; ++j) {
                        const float2 v = sh[(((k - 1) * 2 + c) * kP + j) * 32 + lane];
                        h[c][j] = f2(v.x, v.y);
                    }
            }
            F2 hist[kSub][2][kP];  // states before each row
            float y[kSub][2];
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const uint32_t f = flag(k * kSub + i);
                if (kLook && f != kRowOutside && (f & kRowHead)) load_state(h, p.initial, f & kRowSegment);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int j = 0; j < kP; ++j) hist[i][c][j] = h[c][j];
                y[i][0] = y[i][1] = 0.0f;
                if (kLook && f == kRowOutside) continue;
                step(k * kSub + i, true, y[i]);
            }
#pragma unroll
            for (int i = kSub - 1; i >= 0; --i) {
                const int r = k * kSub + i;
                const uint32_t f = flag(r);
                if (kLook && f == kRowOutside) continue;
                if (kLook && (f & kRowTail)) load_state(e, q.grad_final, f & kRowSegment);
                const float2 d0 = sd[r * kC + own], d1 = sd[r * kC + other];
                const float g0 = sg[r * kC + own], g1 = sg[r * kC + other];
                const F2 dd[2] = {f2(d0.x, d0.x), f2(d1.x, d1.x)}, xx[2] = {f2(d0.y, d0.y), f2(d1.y, d1.y)};
                const F2 dy[2] = {f2(g0, g0), f2(g1, g1)};
                F2 a1[2] = {zero, zero}, a2[2] = {zero, zero}, vb[kP], vc[kP];
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const float2 bv = sbc[r * kN + (n0 / 2 + (j ^ flip))];
                    const float2 cv = sbc[r * kN + kN / 2 + (n0 / 2 + (j ^ flip))];
                    const F2 Bv = f2(bv.x, bv.y), Cv = f2(cv.x, cv.y);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float2 ar = unpack(mul2(dd[c], A2[c][j]));
                        const F2 a = f2(ex2(ar.x), ex2(ar.y));
                        // the state past the row: the next row's, unless that begins a segment
                        const F2 hr = kLook         ? fma2(a, hist[i][c][j], mul2(xx[c], Bv))
                                      : i + 1 < kSub ? hist[i + 1 < kSub ? i + 1 : i][c][j]
                                                     : h[c][j];
                        const F2 dh = fma2(dy[c], Cv, e[c][j]);
                        vc[j] = c ? fma2(dy[c], hr, vc[j]) : mul2(dy[c], hr);
                        vb[j] = c ? fma2(dh, xx[c], vb[j]) : mul2(dh, xx[c]);
                        a1[c] = fma2(dh, Bv, a1[c]);
                        e[c][j] = mul2(dh, a);
                        const F2 w = mul2(e[c][j], hist[i][c][j]);
                        a2[c] = fma2(w, A2[c][j], a2[c]);
                        dA[c][j] = fma2(w, dd[c], dA[c][j]);
                    }
                }
                if (kLook && (f & kRowHead)) {
                    if (q.grad_initial) save_state(q.grad_initial, f & kRowSegment, e);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int j = 0; j < kP; ++j) e[c][j] = zero;
                }
                // over states: this lane's part of its own channel, and the other lane's
                float sums[3][2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float2 v1 = unpack(a1[c]), v2 = unpack(a2[c]);
                    sums[0][c] = v1.x + v1.y, sums[2][c] = y[i][c];
                    sums[1][c] = (v2.x + v2.y) * 0.6931471805599453f;  // A = A2 ln 2
                }
#pragma unroll
                for (int m = 0; m < 3; ++m) {
                    sums[m][0] += __shfl_xor_sync(0xffffffffu, sums[m][1], 1);
#pragma unroll
                    for (int o = 2; o < NL; o <<= 1) sums[m][0] += __shfl_xor_sync(0xffffffffu, sums[m][0], o);
                }
                if (NL == 2 || nl < 2) {
                    s1[r * kC + own] = sums[0][0];
                    s2[r * kC + own] = sums[1][0];
                    sy[r * kC + own] = sums[2][0];
                }
                // over channels: v[which][2 * pair of states + half]
                float v[2][NT];
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const float2 x = unpack(vb[j]), w = unpack(vc[j]);
                    v[0][2 * j] = x.x, v[0][2 * j + 1] = x.y, v[1][2 * j] = w.x, v[1][2 * j + 1] = w.y;
                }
                int left = NT;  // values of each of dB, dC that a lane still holds
#pragma unroll
                for (int s = 0; s < 5; ++s) {  // exchange with the lane whose pair differs in bit s
                    const int o = NL << s;
                    if (o >= 32) break;
                    if (left > 2) {  // the state pairs to keep come first
                        left /= 2;
#pragma unroll
                        for (int w = 0; w < 2; ++w)
#pragma unroll
                            for (int j = 0; j < NT / 2; ++j)
                                if (j < left) v[w][j] += __shfl_xor_sync(0xffffffffu, v[w][j + left], o);
                    } else if (left == 2) {  // one state of the pair
                        const bool up = pair >> s & 1;
#pragma unroll
                        for (int w = 0; w < 2; ++w)
                            v[w][0] = (up ? v[w][1] : v[w][0]) +
                                      __shfl_xor_sync(0xffffffffu, up ? v[w][0] : v[w][1], o);
                        left = 1;
                    } else if (left == 1) {  // dB or dC
                        const bool up = pair >> s & 1;
                        v[0][0] = (up ? v[1][0] : v[0][0]) + __shfl_xor_sync(0xffffffffu, up ? v[0][0] : v[1][0], o);
                        left = 0;
                    } else {
                        v[0][0] += __shfl_xor_sync(0xffffffffu, v[0][0], o);
                    }
                }
                float *to = bc_out + (s0 + r) * bc_row;
                constexpr int kStages = NL == 2 ? 4 : NL == 4 ? 3 : NL == 8 ? 2 : 1;
                constexpr int kHalves = NT == 8 ? 2 : 1;  // exchanges that kept whole state pairs
                if constexpr (kStages > kHalves + 1) {    // one value: dB or dC of one state
                    const int n = n0 + 2 * flip + (pair >> kHalves & 1);
                    const bool first = kStages == kHalves + 2 || (pair >> (kHalves + 2)) == 0;
                    if (first && n < p.states) to[(pair >> (kHalves + 1) & 1) * p.states + n] = v[0][0];
                } else if constexpr (kStages == kHalves + 1) {  // dB and dC of one state
                    const int n = n0 + 2 * flip + (pair >> kHalves & 1);
                    if (n < p.states) to[n] = v[0][0], to[p.states + n] = v[1][0];
                } else {
                    constexpr int kLeft = NT >> kStages;  // values of each
#pragma unroll
                    for (int j = 0; j < kLeft; ++j) {
                        const int n = n0 + 2 * ((j / 2) ^ flip) + j % 2;
                        if (n < p.states) to[n] = v[0][j], to[p.states + n] = v[1][j];
                    }
                }
            }
        }
    };

    const int64_t last = t0 + (t1 - 1 - t0) / kTile * kTile;
#pragma unroll 1
    for (int64_t s0 = last; s0 >= t0; s0 -= kTile) {
        const int rows = int(min(int64_t(kTile), t1 - s0));
        uint32_t code = kRowOutside;
        if (lane < rows) code = p.segmap ? p.segmap[s0 + lane] : 0u;
        const bool plain = __all_sync(0xffffffffu, lane >= kTile || (code & (kRowHead | kRowTail)) == 0u);
        if (s0 - kTile >= t0) {  // ask L2 for the rows of the next tile, and the state before it
            const int64_t t = s0 - kTile + lane % kTile;
            prefetch_l2(lane < kTile ? dt + t * p.dt_row : u + t * p.u_row);
            prefetch_l2(lane < kTile ? z + t * z_row : go + t * q.grad_row);
            prefetch_l2(lane < kTile ? B + t * p.b_row : C + t * p.c_row);
            const float *x = p.checkpoints +
                             ((int64_t(b) * p.tiles + s0 / kTile - 1) * p.channels + cb) * p.states;
            for (int i = lane * 32; i < live * p.states; i += 32 * 32) prefetch_l2(x + i);
        }
        // rows past the last are read as the last, and not used
#pragma unroll 8
        for (int m = 0; m < kMine; ++m) {
            const int r = mine_row + m * kMineRows;
            const int64_t t = min(s0 + r, t1 - 1);
            float d = to_f32<T>((dt + t * p.dt_row)[mine_at]) + bias;
            if (p.softplus) d = softplus_poly(d);
            const float x = d * to_f32<T>((u + t * p.u_row)[mine_at]);
            float dy = to_f32<T>((go + t * q.grad_row)[mine_at]);
            const float zv = to_f32<T>((z + t * z_row)[mine_at]);
            if (p.z) dy *= silu(zv);
            // a channel past the last adds nothing to dB and dC
            sd[r * kC + mine] = mine < live ? make_float2(d, x) : make_float2(0.0f, 0.0f);
            sg[r * kC + mine] = mine < live ? dy : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kTile * kN / 32; ++i) {
            const int at = lane + 32 * i, r = at / kN, n = at % kN;
            const int64_t t = min(s0 + r, t1 - 1);
            const int m = min(n, p.states - 1);
            const float bv = to_f32<T>(B[t * p.b_row + m]), cv = to_f32<T>(C[t * p.c_row + m]);
            float *to = reinterpret_cast<float *>(sbc) + r * 2 * kN + n;
            to[0] = n < p.states ? bv : 0.0f;
            to[kN] = n < p.states ? cv : 0.0f;
        }
        __syncwarp();
        if (plain) tile(s0, rows, code, std::false_type());
        else tile(s0, rows, code, std::true_type());
        __syncwarp();
        // loads of several rows before the first store, which would hold them back
        constexpr int kBatch = kMine < 8 ? kMine : 8;
#pragma unroll 1
        for (int m0 = 0; m0 < kMine; m0 += kBatch) {
            T ru[kBatch], rd[kBatch], rz[kBatch], rg[kBatch];
#pragma unroll
            for (int m = 0; m < kBatch; ++m) {
                const int64_t t = min(s0 + mine_row + (m0 + m) * kMineRows, t1 - 1);
                ru[m] = (u + t * p.u_row)[mine_at];
                rd[m] = (dt + t * p.dt_row)[mine_at];
                rz[m] = (z + t * z_row)[mine_at];
                rg[m] = (go + t * q.grad_row)[mine_at];
            }
#pragma unroll
            for (int m = 0; m < kBatch; ++m) {
                const int r = mine_row + (m0 + m) * kMineRows;
                const uint32_t f = __shfl_sync(0xffffffffu, code, r);
                const int64_t t = s0 + r;
                const float uv = to_f32<T>(ru[m]), q1 = s1[r * kC + mine], dy = sg[r * kC + mine];
                float dd = fmaf(q1, uv, s2[r * kC + mine]);
                if (p.softplus) dd *= sigmoid(to_f32<T>(rd[m]) + bias);  // the slope of softplus
                const float du = fmaf(q1, sd[r * kC + mine].x, Dv * dy);
                const float zv = to_f32<T>(rz[m]);
                const float dz = to_f32<T>(rg[m]) * fmaf(Dv, uv, sy[r * kC + mine]) * silu_slope(zv, sigmoid(zv));
                if (mine < live && f != kRowOutside) {
                    gu[t * p.channels + mine] = from_f32<T>(du);
                    gdt[t * p.channels + mine] = from_f32<T>(dd);
                    if (p.z) gz[t * p.channels + mine] = from_f32<T>(dz);
                    acc_D = fmaf(dy, uv, acc_D);
                    acc_bias += dd;
                }
            }
        }
        __syncwarp();
    }
    if (!p.segmap && t0 == 0 && q.grad_initial) save_state(q.grad_initial, b, e);

    // the parameters' shares of this block: [dA | dD | ddt_bias]
    float *part = q.partial + int64_t(blockIdx.x) * p.channels * (p.states + 2);
    save_state(part, 0, dA);
#pragma unroll
    for (int o = kC; o < 32; o <<= 1) {
        acc_D += __shfl_xor_sync(0xffffffffu, acc_D, o);
        acc_bias += __shfl_xor_sync(0xffffffffu, acc_bias, o);
    }
    if (lane < live) {
        part[p.channels * p.states + cb + lane] = acc_D;
        part[p.channels * (p.states + 1) + cb + lane] = acc_bias;
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
#pragma unroll 8
    for (uint32_t k = 0; k < p.group_blocks; ++k) s += q.partial_bc[k * total + i];
    const int64_t at = i % per, g = at / (2 * p.states), which = at / p.states % 2, n = at % p.states;
    T *to = static_cast<T *>(which ? q.grad_C : q.grad_B);
    to[(row * p.groups + g) * p.states + n] = from_f32<T>(s);
}

template <class T, int NT, int NL>
cudaError_t backward_v(ScanBackwardParams q, cudaStream_t s) {
    ScanParams &p = q.f;
    constexpr int kC = 64 / NL;
    p.group_blocks = uint32_t((p.group + kC - 1) / kC);
    const dim3 grid(uint32_t(p.batch * p.chunks), uint32_t(p.groups * p.group_blocks));
    cudaError_t err = launch_pdl(selscan_backward_kernel<T, NT, NL>, grid, dim3(32), 0, s, q);
    if (err != cudaSuccess) return err;
    const int64_t total = int64_t(p.batch) * p.rows * p.groups * 2 * p.states;
    return launch_pdl(join_bc_kernel<T>, dim3(uint32_t((total + 255) / 256)), dim3(256), 0, s, q, total);
}

template <class T>
cudaError_t backward_t(const ScanBackwardParams &q, cudaStream_t s) {
    const int n = q.f.states;
    if (n <= 8) return backward_v<T, 4, 2>(q, s);
    if (n <= 16) return backward_v<T, 8, 2>(q, s);
    if (n <= 32) return backward_v<T, 8, 4>(q, s);
    if (n <= 64) return backward_v<T, 8, 8>(q, s);
    return backward_v<T, 8, 16>(q, s);
}

}  // namespace

}  // namespace dwp
