// Building blocks of the sequence operators (causal convolution, selective
// scan, block norm): element types, loads and stores of a few neighbouring
// channels, the smooth functions, and the walk over packed segments.
//
// Rows are tokens and the channels of a row are contiguous, so a thread takes
// V neighbouring channels: V elements fill 16 bytes (or 8) where every row
// of the tensor starts on such a boundary, and V = 1 serves every other
// stride, base or odd channel count.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device.cuh"
#include "launch.h"

namespace dwp {

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// V elements moved as one access; V * sizeof(T) is 2, 4, 8, 16 or 32 bytes.
template <class T, int V>
struct alignas((V * sizeof(T)) < 16 ? V * sizeof(T) : 16) Pack {
    T e[V];
};

template <int V, class T>
__device__ __forceinline__ void load_f32(float (&f)[V], const T *p) {
    const Pack<T, V> r = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32<T>(r.e[i]);
}

template <int V, class T>
__device__ __forceinline__ void store_f32(T *p, const float (&f)[V]) {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.e[i] = from_f32<T>(f[i]);
    *reinterpret_cast<Pack<T, V> *>(p) = r;
}

// A parameter held in f32 or in the activations' type.
template <class T>
__device__ __forceinline__ float load_param(const void *p, uint64_t i, bool is_f32) {
    return is_f32 ? static_cast<const float *>(p)[i] : to_f32<T>(static_cast<const T *>(p)[i]);
}

// V neighbouring parameters from i on, as one access.
template <class T, int V>
__device__ __forceinline__ void load_params(float (&f)[V], const void *p, uint64_t i, bool is_f32) {
    if (is_f32) load_f32<V>(f, static_cast<const float *>(p) + i);
    else load_f32<V>(f, static_cast<const T *>(p) + i);
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Logistic function 1 / (1 + e^-x); for large -x the exponential is +inf and
// the quotient 0, the limit.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.0f + ex2(x * -kLog2e)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
// d/dx of x * sigmoid(x), from x and s = sigmoid(x).
__device__ __forceinline__ float silu_slope(float x, float s) { return s * fmaf(x, 1.0f - s, 1.0f); }

// Two f32 in one 64-bit register pair.  One packed instruction does two
// multiply-adds at the same rate as two scalar ones but takes one issue slot
// (measured: 2.1-2.4 cycles a warp and scheduler against 1.04 each).
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// acc += a * b of V values, in pairs where V is even.
template <int V>
__device__ __forceinline__ void fma_to(float (&acc)[V], const float (&a)[V], const float (&b)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 r = unpack(fma2(f2(a[i], a[i + 1]), f2(b[i], b[i + 1]), f2(acc[i], acc[i + 1])));
            acc[i] = r.x, acc[i + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(a[i], b[i], acc[i]);
    }
}

// Segment of packed row `t` by CSR offsets (num_segments + 1 entries): the
// first s with offsets[s + 1] > t, or num_segments if there is none.  Empty
// segments are passed over.  Any offsets give s <= num_segments.
__device__ __forceinline__ uint32_t segment_of(const uint32_t *offsets, uint32_t num_segments,
                                               uint32_t t) {
    uint32_t lo = 0, hi = num_segments;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2u;
        if (offsets[mid + 1] > t) hi = mid;
        else lo = mid + 1u;
    }
    return lo;
}

}  // namespace dwp
