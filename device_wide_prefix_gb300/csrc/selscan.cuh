// Building blocks of the selective scan's kernels: packed f32 pairs, the
// smooth functions of a row's step, and the rows' staging.
#pragma once

#include <type_traits>

#include "sequence.cuh"

namespace dwp {

constexpr int kCheckpointRows = DWP_SCAN_CHECKPOINT_ROWS;

// Code words of the segment map.
constexpr uint32_t kRowHead = 0x80000000u;
constexpr uint32_t kRowTail = 0x40000000u;
constexpr uint32_t kRowSegment = 0x3fffffffu;
constexpr uint32_t kRowOutside = 0xffffffffu;

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

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// log(1 + e^x) = max(x, 0) + log1p(e^-|x|).  log1p(e) / e on [0, 1] is a
// degree-8 polynomial fitted for the least relative error (3.0e-8; 1.8e-7
// evaluated in f32); with the exponential's own error the result is within
// 5e-7 for |x| < 16.  12 instructions, where log1pf(expf(x)) took about 40.
// Scalar on purpose: its constants are immediates, which packed instructions
// do not take.
__device__ __forceinline__ float softplus_poly(float x) {
    const float e = ex2(-fabsf(x) * kLog2e);
    float p = 0.0052326880395412445f;
    p = fmaf(p, e, -0.029505213722586632f);
    p = fmaf(p, e, 0.07822591066360474f);
    p = fmaf(p, e, -0.13663242757320404f);
    p = fmaf(p, e, 0.19106005132198334f);
    p = fmaf(p, e, -0.2484298199415207f);
    p = fmaf(p, e, 0.3331909775733948f);
    p = fmaf(p, e, -0.4999949336051941f);
    p = fmaf(p, e, 0.9999999403953552f);
    return fmaf(p, e, fmaxf(x, 0.0f));
}

}  // namespace dwp
