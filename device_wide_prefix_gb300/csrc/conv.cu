// Short causal depthwise convolution over packed rows: forward, gradient and
// the single-token form.
//
//   p[t] = bias + sum_k w[k] x[t - (W-1) + k],   y = p or p * sigmoid(p)
//
// per channel, where rows before a segment's first come from its state rows.
// Every element is read and written once: the work is HBM traffic.
#include <type_traits>

#include "sequence.cuh"

namespace dwp {

namespace {

// Every kernel below is made for its width W.  One for widths up to W, with
// taps of 0 past the width, would multiply rows that the definition does not
// reach, and 0 times an infinity there is NaN.

constexpr int kConvThreads = 128;
constexpr int kConvStrip = 64;  // rows one thread walks

// Where a packed row lies: its segment and the segment's rows.
struct Span {
    uint32_t seg;
    int64_t begin, end;  // rows [begin, end) of this batch entry's stream
};

// Segment span at row t (packed: by offsets; otherwise the whole batch entry).
// A row that no segment covers gets begin > t.
__device__ __forceinline__ Span span_at(const uint32_t *offsets, uint32_t nseg, uint32_t batch,
                                        int64_t rows, int64_t t) {
    if (!offsets) return {batch, 0, rows};
    const uint32_t s = segment_of(offsets, nseg, static_cast<uint32_t>(t));
    if (s >= nseg) return {s, rows, rows};
    return {s, int64_t(offsets[s]), min(int64_t(offsets[s + 1]), rows)};
}

// Taps and bias of V channels: w[j][i] is channel i's for j rows before the
// row itself.
template <class T, int V, int W, class Params>
__device__ __forceinline__ void load_taps(const Params &p, int64_t c0, float (&w)[W][V], float (&bias)[V]) {
    if (W == 4 && p.weight_f32 && p.weight_wide) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(p.weight)[c0 + i];
            const float taps[4] = {v.w, v.z, v.y, v.x};
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = taps[j % 4];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j)
                w[j][i] = load_param<T>(p.weight, (c0 + i) * W + (W - 1 - j), p.weight_f32);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = p.bias ? load_param<T>(p.bias, c0 + i, p.weight_f32) : 0.0f;
}

// The W - 1 inputs before row t of span `sp`: win[j - 1] is row t - j, or the
// state row that stands for it.
template <class T, int V, int W>
__device__ __forceinline__ void load_window(const ConvParams &p, const Span &sp, const T *x, int64_t t, int64_t c0,
                                            float (&win)[W][V]) {
    constexpr int halo = W - 1;
    const T *init = static_cast<const T *>(p.initial_state);
#pragma unroll
    for (int j = 1; j < W; ++j) {
        const int64_t r = t - j;
#pragma unroll
        for (int i = 0; i < V; ++i) win[j - 1][i] = 0.0f;
        if (r >= sp.begin) load_f32<V>(win[j - 1], x + r * p.x_row);
        else if (init)
            load_f32<V>(win[j - 1], init + (int64_t(sp.seg) * halo + (r - sp.begin + halo)) * p.channels + c0);
    }
}

template <int V, int W>
__device__ __forceinline__ void push(float (&win)[W][V], const float (&x)[V]) {
#pragma unroll
    for (int j = W - 1; j > 0; --j)
#pragma unroll
        for (int i = 0; i < V; ++i) win[j][i] = win[j - 1][i];
#pragma unroll
    for (int i = 0; i < V; ++i) win[0][i] = x[i];
}

constexpr int kConvGroup = 4;  // rows loaded together, one group ahead of their use

// Forward.  A thread walks kConvStrip rows of V channels with the last W - 1
// inputs and the taps in registers, so each input is read once (plus W - 1
// rows per strip).  Four 16-bit channels a thread and 85 registers (24 warps an
// SM) carry 16384 x 5120 bf16 in 82 us, 97 warp instructions a row, issue 0.71 a
// cycle; without the prefetch it took 3 us more, with eight channels and 12
// warps 22, with 64 registers 29.
template <class T, int V, int W>
__global__ void __launch_bounds__(kConvThreads, W <= 4 ? 6 : 2) conv_kernel(ConvParams p) {
    pdl_trigger();
    pdl_wait();
    const int64_t c0 = (int64_t(blockIdx.y) * kConvThreads + threadIdx.x) * V;
    if (c0 >= p.channels) return;
    const uint32_t b = blockIdx.x / p.strips;
    const int64_t t0 = int64_t(blockIdx.x % p.strips) * kConvStrip;
    const int64_t t1 = min(t0 + kConvStrip, p.rows);
    constexpr int halo = W - 1;
    const T *x = static_cast<const T *>(p.x) + int64_t(b) * p.x_batch + c0;
    T *y = static_cast<T *>(p.y) + int64_t(b) * p.y_batch + c0;
    T *fin = static_cast<T *>(p.final_state);

    Pack<T, V> next[kConvGroup];
    auto load = [&](int64_t t) {  // rows past the last are read as the last
#pragma unroll
        for (int i = 0; i < kConvGroup; ++i)
            next[i] = *reinterpret_cast<const Pack<T, V> *>(x + min(t + i, t1 - 1) * p.x_row);
        // the registers hold too few rows in flight for HBM: the group after
        // this one is on its way to L2
#pragma unroll
        for (int i = 0; i < kConvGroup; ++i)
            if (t + kConvGroup + i < t1) prefetch_l2(x + (t + kConvGroup + i) * p.x_row);
    };
    load(t0);
    float w[W][V], bias[V], win[W][V];
    load_taps<T, V, W>(p, c0, w, bias);
    Span sp{0, p.rows, 0};
    for (int64_t s = t0; s < t1; s += kConvGroup) {
        Pack<T, V> now[kConvGroup];
#pragma unroll
        for (int i = 0; i < kConvGroup; ++i) now[i] = next[i];
        if (s + kConvGroup < t1) load(s + kConvGroup);
        auto row = [&](int64_t t, const Pack<T, V> &xv) {
            float o[V];
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = to_f32<T>(xv.e[k]);
            push<V, W>(win, o);
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = bias[k];
#pragma unroll
            for (int j = 0; j < W; ++j) fma_to<V>(o, w[j], win[j]);
            if (p.silu) {
#pragma unroll
                for (int k = 0; k < V; ++k) o[k] = silu(o[k]);
            }
            store_f32<V>(y + t * p.y_row, o);
        };
        // inside one segment, and past its first row: that one loads the window
        if (s > t0 && s + kConvGroup <= t1 && sp.begin < s && s + kConvGroup < sp.end) {
#pragma unroll
            for (int i = 0; i < kConvGroup; ++i) row(s + i, now[i]);
            continue;
        }
#pragma unroll 1
        for (int64_t t = s; t < min(s + kConvGroup, t1); ++t) {
            if (t == t0 || t == sp.begin || t >= sp.end) {  // also the first row after rows outside
                sp = span_at(p.offsets, p.num_segments, b, p.rows, t);
                if (sp.begin <= t) load_window<T, V, W>(p, sp, x, t, c0, win);
            }
            if (sp.begin <= t) {  // else outside every segment: left unwritten
                row(t, now[0]);
                if (fin && t == sp.end - 1) {
#pragma unroll
                    for (int j = 0; j < halo; ++j)
                        store_f32<V>(fin + (int64_t(sp.seg) * halo + (halo - 1 - j)) * p.channels + c0, win[j]);
                }
            }
#pragma unroll
            for (int i = 0; i + 1 < kConvGroup; ++i) now[i] = now[i + 1];
        }
    }
}

// An empty segment hands its state on: dst rows = src rows (0 without src).
template <class T>
__global__ void __launch_bounds__(kConvThreads)
    empty_state_kernel(const uint32_t *offsets, int64_t count, const T *src, T *dst) {
    pdl_trigger();
    pdl_wait();
    const int64_t s = blockIdx.x;
    if (offsets && offsets[s] < offsets[s + 1]) return;
    for (int64_t i = int64_t(blockIdx.y) * kConvThreads + threadIdx.x; i < count; i += int64_t(gridDim.y) * kConvThreads)
        dst[s * count + i] = src ? src[s * count + i] : from_f32<T>(0.0f);
}

// Gradient.  With g[t] = dy[t] * act'(p[t]), each tap scatters g backwards:
// row t - j of the segment (or the state row that stands for it) receives
// w[W-1-j] g[t].  A thread walks its strip and W - 1 rows past it with the
// unfinished sums in registers, and writes a row's sum once the last tap
// reached it.  Each row's g also adds to the taps' gradients, which a thread
// sums over its strip and a second kernel over the strips, in a fixed order.
// 4 x 2048 x 4096 bf16: 201 MB in 74 us, 11 of them the second kernel (92 when
// one kernel served every width up to four); 94 warp instructions a row, issue
// 0.64 a cycle.  Two channels a thread and 28 warps an SM; four and 16 took 11
// us more.
template <class T, int V, int W>
__global__ void __launch_bounds__(kConvThreads, W <= 4 ? 7 : 3) conv_backward_kernel(ConvBackwardParams q) {
    pdl_trigger();
    pdl_wait();
    const ConvParams &p = q.c;
    const int64_t c0 = (int64_t(blockIdx.y) * kConvThreads + threadIdx.x) * V;
    if (c0 >= p.channels) return;
    const uint32_t b = blockIdx.x / p.strips;
    const int64_t t0 = int64_t(blockIdx.x % p.strips) * q.strip_rows;
    const int64_t t1 = min(t0 + q.strip_rows, p.rows);
    constexpr int halo = W - 1;
    const int64_t te = min(t1 + halo, p.rows);

    const T *x = static_cast<const T *>(p.x) + int64_t(b) * p.x_batch + c0;
    const T *dy = static_cast<const T *>(q.grad_out) + int64_t(b) * q.grad_batch + c0;
    T *dx = static_cast<T *>(q.grad_x) + int64_t(b) * q.gx_batch + c0;
    T *dinit = static_cast<T *>(q.grad_initial);
    const T *dfin = static_cast<const T *>(q.grad_final);

    Pack<T, V> nx[kConvGroup], ng[kConvGroup];
    auto load = [&](int64_t t) {  // rows past the last are read as the last
#pragma unroll
        for (int i = 0; i < kConvGroup; ++i) {
            const int64_t r = min(t + i, te - 1);
            nx[i] = *reinterpret_cast<const Pack<T, V> *>(x + r * p.x_row);
            ng[i] = *reinterpret_cast<const Pack<T, V> *>(dy + r * q.grad_row);
        }
    };
    load(t0);
    float w[W][V], bias[V];
    load_taps<T, V, W>(p, c0, w, bias);
    float win[W][V], acc[W][V], dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = acc[j][i] = win[j][i] = 0.0f;
    }
    Span sp{0, p.rows, 0};
    // the finished sum of row r: an own row of the strip, or a state row of a
    // segment that begins in the strip
    auto put = [&](int64_t r, const float(&v)[V]) {
        if (r >= sp.begin) {
            if (r >= t0 && r < t1) store_f32<V>(dx + r * q.gx_row, v);
        } else if (dinit && sp.begin >= t0 && sp.begin < t1 && r >= sp.begin - halo) {
            store_f32<V>(dinit + (int64_t(sp.seg) * halo + (r - sp.begin + halo)) * p.channels + c0, v);
        }
    };
    bool over = false;  // a segment of the next strip begins
    for (int64_t s = t0; s < te && !over; s += kConvGroup) {
        Pack<T, V> cx[kConvGroup], cg[kConvGroup];
#pragma unroll
        for (int i = 0; i < kConvGroup; ++i) cx[i] = nx[i], cg[i] = ng[i];
        if (s + kConvGroup < te) load(s + kConvGroup);
        // row t: its p and g, and what g adds to the rows and taps; `mine`: a row of this strip
        auto row = [&](const Pack<T, V> &xr, const Pack<T, V> &gr, bool mine) {
            float xv[V], g[V], none[V];
#pragma unroll
            for (int k = 0; k < V; ++k) xv[k] = to_f32<T>(xr.e[k]), g[k] = to_f32<T>(gr.e[k]), none[k] = 0.0f;
            push<V, W>(win, xv);
            push<V, W>(acc, none);
            if (p.silu) {
                float a[V];
#pragma unroll
                for (int k = 0; k < V; ++k) a[k] = bias[k];
#pragma unroll
                for (int j = 0; j < W; ++j) fma_to<V>(a, w[j], win[j]);
#pragma unroll
                for (int k = 0; k < V; ++k) g[k] *= silu_slope(a[k], sigmoid(a[k]));
            }
#pragma unroll
            for (int j = 0; j < W; ++j) fma_to<V>(acc[j], w[j], g);
            if (mine) {
#pragma unroll
                for (int k = 0; k < V; ++k) db[k] += g[k];
#pragma unroll
                for (int j = 0; j < W; ++j) fma_to<V>(dw[j], g, win[j]);
            }
        };
        if (s - halo >= t0 && s + kConvGroup <= t1 && sp.begin <= s - halo && s + kConvGroup < sp.end) {
            // inside one segment, and every finished row is this strip's
#pragma unroll
            for (int i = 0; i < kConvGroup; ++i) {
                row(cx[i], cg[i], true);
                store_f32<V>(dx + (s + i - halo) * q.gx_row, acc[halo]);
            }
            continue;
        }
#pragma unroll 1
        for (int64_t t = s; t < min(s + kConvGroup, te); ++t) {
            if (t == t0 || t == sp.begin || t >= sp.end) {  // also the first row after rows outside
                sp = span_at(p.offsets, p.num_segments, b, p.rows, t);
                if (sp.begin <= t) {
                    if (t >= t1 && sp.begin == t) {
                        over = true;
                        break;
                    }
                    load_window<T, V, W>(p, sp, x, t, c0, win);
#pragma unroll
                    for (int j = 0; j < W; ++j)
#pragma unroll
                        for (int k = 0; k < V; ++k) acc[j][k] = 0.0f;
                }
            }
            if (sp.begin <= t) {
                row(cx[0], cg[0], t < t1);
                put(t - halo, acc[halo]);
                if (t == sp.end - 1) {  // the rows that no later row of the segment reaches
#pragma unroll
                    for (int j = 0; j < halo; ++j) {
                        float v[V];
#pragma unroll
                        for (int k = 0; k < V; ++k) v[k] = 0.0f;
                        if (dfin) load_f32<V>(v, dfin + (int64_t(sp.seg) * halo + (halo - 1 - j)) * p.channels + c0);
#pragma unroll
                        for (int k = 0; k < V; ++k) v[k] += acc[j][k];
                        put(t - j, v);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i + 1 < kConvGroup; ++i) cx[i] = cx[i + 1], cg[i] = cg[i + 1];
        }
    }
    float *part = q.partial + (int64_t(blockIdx.x) * (W + 1)) * p.channels + c0;
#pragma unroll
    for (int j = 0; j < W; ++j) store_f32<V>(part + int64_t(halo - j) * p.channels, dw[j]);
    store_f32<V>(part + int64_t(W) * p.channels, db);
}

// One token for each row of a batch: the slot's W - 1 state rows and the new
// input give the output, and the state moves on by one row.
template <class T, int V, int W>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvStepParams p) {
    pdl_trigger();
    pdl_wait();
    const int64_t c0 = (int64_t(blockIdx.y) * kConvThreads + threadIdx.x) * V;
    if (c0 >= p.channels) return;
    const int64_t b = blockIdx.x;
    constexpr int halo = W - 1;
    T *y = static_cast<T *>(p.y) + b * p.y_row + c0;
    const int64_t slot = p.slots ? p.slots[b] : b;
    const bool live = slot >= 0 && slot < p.num_slots;  // else a padding row
    // the taps do not wait for the slot
    float w[W][V], o[V], win[W][V];
    load_taps<T, V, W>(p, c0, w, o);
    T *st = static_cast<T *>(p.state) + (live ? slot : 0) * p.state_slot + c0;
    load_f32<V>(win[0], static_cast<const T *>(p.x) + b * p.x_row + c0);
#pragma unroll
    for (int j = 1; j < W; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) win[j][i] = 0.0f;
        if (live) load_f32<V>(win[j], st + int64_t(halo - j) * p.channels);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) o[i] = fmaf(w[j][i], win[j][i], o[i]);
        if (p.silu) o[i] = silu(o[i]);
        if (!live) o[i] = 0.0f;
    }
    store_f32<V>(y, o);
    if (!live) return;
#pragma unroll
    for (int j = 0; j < halo; ++j) store_f32<V>(st + int64_t(halo - 1 - j) * p.channels, win[j]);
}

// go(W) for W = width, which the entry points hold to 1 .. 8.
template <class F>
cudaError_t by_width(int width, F go) {
    switch (width) {
        case 1: return go(std::integral_constant<int, 1>());
        case 2: return go(std::integral_constant<int, 2>());
        case 3: return go(std::integral_constant<int, 3>());
        case 4: return go(std::integral_constant<int, 4>());
        case 5: return go(std::integral_constant<int, 5>());
        case 6: return go(std::integral_constant<int, 6>());
        case 7: return go(std::integral_constant<int, 7>());
        case 8: return go(std::integral_constant<int, 8>());
    }
    return cudaErrorInvalidValue;
}

template <class T, int V>
cudaError_t conv_forward_w(const ConvParams &p, cudaStream_t s) {
    const dim3 grid(uint32_t(p.batch * p.strips), uint32_t((p.channels + kConvThreads * V - 1) / (kConvThreads * V)));
    return by_width(p.width, [&](auto w) {
        return launch_pdl(conv_kernel<T, V, decltype(w)::value>, grid, dim3(kConvThreads), 0, s, p);
    });
}

template <class T, int V>
cudaError_t conv_backward_w(const ConvBackwardParams &q, cudaStream_t s) {
    const ConvParams &p = q.c;
    const dim3 grid(uint32_t(p.batch * p.strips), uint32_t((p.channels + kConvThreads * V - 1) / (kConvThreads * V)));
    return by_width(p.width, [&](auto w) {
        return launch_pdl(conv_backward_kernel<T, V, decltype(w)::value>, grid, dim3(kConvThreads), 0, s, q);
    });
}

template <class T, int V>
cudaError_t conv_step_w(const ConvStepParams &p, cudaStream_t s) {
    const dim3 grid(uint32_t(p.batch), uint32_t((p.channels + kConvThreads * V - 1) / (kConvThreads * V)));
    return by_width(p.width, [&](auto w) {
        return launch_pdl(conv_step_kernel<T, V, decltype(w)::value>, grid, dim3(kConvThreads), 0, s, p);
    });
}

template <class T>
cudaError_t empty_states(const uint32_t *offsets, int64_t segments, int64_t count, const void *src, void *dst,
                         cudaStream_t s) {
    const int64_t spread = (count + kConvThreads - 1) / kConvThreads;  // few segments: many blocks to each
    const uint32_t per = uint32_t(segments >= 1024 ? 1 : spread < 1024 / segments ? spread : 1024 / segments);
    return launch_pdl(empty_state_kernel<T>, dim3(uint32_t(segments), per), dim3(kConvThreads), 0, s, offsets, count,
                      static_cast<const T *>(src), static_cast<T *>(dst));
}

}  // namespace

int64_t conv_strip_rows() { return kConvStrip; }

cudaError_t launch_empty_states(dwp_dtype t, const uint32_t *offsets, int64_t segments, int64_t count,
                                const void *src, void *dst, cudaStream_t s) {
    if (segments == 0 || count == 0) return cudaSuccess;
    if (t == DWP_F32) return empty_states<float>(offsets, segments, count, src, dst, s);
    if (t == DWP_BF16) return empty_states<__nv_bfloat16>(offsets, segments, count, src, dst, s);
    return empty_states<__half>(offsets, segments, count, src, dst, s);
}

cudaError_t launch_conv(dwp_dtype t, const ConvParams &p, bool vec, cudaStream_t s) {
    if (t == DWP_F32) return vec ? conv_forward_w<float, 4>(p, s) : conv_forward_w<float, 1>(p, s);
    if (t == DWP_BF16) return vec ? conv_forward_w<__nv_bfloat16, 4>(p, s) : conv_forward_w<__nv_bfloat16, 1>(p, s);
    return vec ? conv_forward_w<__half, 4>(p, s) : conv_forward_w<__half, 1>(p, s);
}

cudaError_t launch_conv_backward(dwp_dtype t, const ConvBackwardParams &p, bool vec, cudaStream_t s) {
    if (t == DWP_F32) return vec ? conv_backward_w<float, 2>(p, s) : conv_backward_w<float, 1>(p, s);
    if (t == DWP_BF16)
        return vec ? conv_backward_w<__nv_bfloat16, 2>(p, s) : conv_backward_w<__nv_bfloat16, 1>(p, s);
    return vec ? conv_backward_w<__half, 2>(p, s) : conv_backward_w<__half, 1>(p, s);
}

cudaError_t launch_conv_step(dwp_dtype t, const ConvStepParams &p, bool vec, cudaStream_t s) {
    if (t == DWP_F32) return vec ? conv_step_w<float, 2>(p, s) : conv_step_w<float, 1>(p, s);
    if (t == DWP_BF16) return vec ? conv_step_w<__nv_bfloat16, 2>(p, s) : conv_step_w<__nv_bfloat16, 1>(p, s);
    return vec ? conv_step_w<__half, 2>(p, s) : conv_step_w<__half, 1>(p, s);
}

}  // namespace dwp
