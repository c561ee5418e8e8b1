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

// A log2(e), held to finite values.  Past |A| = 2.4e38 it would be infinite,
// and 0 times that (a delta of 0; a lane past the last channel) NaN, where
// exp(0 A) is 1.
__device__ __forceinline__ float decay_rate(float A) {
    float r;  // the forms that hand a NaN on; a test of the infinite cost the scan 4%
    asm("{.reg .f32 t; max.NaN.f32 t, %1, 0fFF7FFFFF; min.NaN.f32 %0, t, 0f7F7FFFFF;}" : "=f"(r) : "f"(A * kLog2e));
    return r;
}
__device__ __forceinline__ F2 decay_rate(F2 A) {
    const float2 v = unpack(A);
    return f2(decay_rate(v.x), decay_rate(v.y));
}

// log(1 + e^x) = max(x, 0) + log1p(e^-|x|).  log1p(e) / e on [0, 1] is a
// degree-8 polynomial fitted for the least relative error (3.0e-8; 1.8e-7
// evaluated in f32).  For x < 0 the rounding of |x| log2(e) adds up to 7.4e-8
// |x|.  Measured, relative: 2.6e-7 on [-4, 0], 7.4e-7 on [-12, -4], 1.7e-6 on
// [-40, -16], 3.6e-6 on [-80, -40], 1.7e-7 for x > 0.  12 instructions, where
// log1pf(expf(x)) took about 40.
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
