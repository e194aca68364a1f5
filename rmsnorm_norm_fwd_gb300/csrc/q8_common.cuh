// q8_common.cuh -- what the kernels of the 8-bit operators share: the code
// arithmetic, and maxima that keep a NaN.
#pragma once

#include "ex_kernels.cuh"
#include "q8_params.h"

namespace gbn {

// Groups whose values all lie below this are stored as zeros with scale 0 (a
// scale this small has no normal fp32 reciprocal to multiply by).
constexpr float kQ8Tiny = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ float q8_max(int fmt) { return fmt == kI8 ? 127.f : 448.f; }
__device__ __forceinline__ float q8_inv_max(int fmt) { return fmt == kI8 ? 1.f / 127.f : 1.f / 448.f; }

// Maximum / minimum that return NaN if either operand is NaN, so that a NaN
// anywhere in a group reaches the group's scale.
__device__ __forceinline__ float fmax_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float fmin_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Q / amax, 0 for a group of zeros (NaN stays NaN).
__device__ __forceinline__ float q8_inv(float amax, float qmax) {
    return amax < kQ8Tiny ? 0.f : __fdiv_rn(qmax, amax);
}
// amax * mul / Q rounded as the division rounds it, so that every kernel writes
// the bits of the definition: the product with the rounded reciprocal, corrected
// by its exact remainder (Markstein 1990).  Tried for every fp32 dividend and both
// Q: only subnormal quotients by 448 may differ, in their last place.  1024 x
// 65536 with group scales 48.7 us, 48.4 us without the correction, 49.4 us with
// the division and its branch.  An infinite amax gives NaN.  A group of zeros: 0,
// also beside an infinite mul (rstd of a row of zeros with eps 0), but NaN with a
// NaN one (a NaN elsewhere in the row).
__device__ __forceinline__ float q8_scale(float amax, float mul, float qmax, float inv_qmax) {
    const float a = amax * mul, q = a * inv_qmax;
    return amax < kQ8Tiny ? fmin_nan(mul, 0.f) : __fmaf_rn(__fmaf_rn(-q, qmax, a), inv_qmax, q);
}

// Two e4m3 codes (low byte: a), saturating at +-448, nearest even.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// Two e4m3 codes widened to fp32 (exact).
__device__ __forceinline__ float2 e4m3_to_f2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// rint(u) for |u| <= 127 as a byte: adding 1.5 * 2^23 rounds to nearest even
// and leaves the two's complement integer in the low byte.
__device__ __forceinline__ uint32_t i8_code(float u) { return __float_as_uint(__fadd_rn(u, 12582912.f)) & 0xffu; }

__device__ __forceinline__ uint8_t q8_code(float u, int fmt) {
    return fmt == kI8 ? (uint8_t)i8_code(u) : (uint8_t)e4m3_pair(u, 0.f);
}
__device__ __forceinline__ float q8_value(uint8_t code, int fmt) {
    return fmt == kI8 ? (float)(int8_t)code : e4m3_to_f2(code).x;
}

// The checkpoint's group: (scale, mid) and the reciprocal used for the codes.
// Plain fp32 steps in this order: the codes depend on the rows alone, so
// every kernel writes the same bits.
struct CkGroup {
    float scale, mid, inv;
};
__device__ __forceinline__ CkGroup ck_group(float top, float low) {
    CkGroup g;
    g.mid = __fadd_rn(__fmul_rn(top, 0.5f), __fmul_rn(low, 0.5f));
    const float half = fmax_nan(__fsub_rn(top, g.mid), __fsub_rn(g.mid, low));
    g.scale = half < kQ8Tiny ? 0.f : __fdiv_rn(half, 127.f);
    g.inv = half < kQ8Tiny ? 0.f : __fdiv_rn(1.f, g.scale);
    return g;
}
__device__ __forceinline__ uint32_t ck_code(float h, const CkGroup &g) {
    return i8_code(__fmul_rn(__fsub_rn(h, g.mid), g.inv));
}

}  // namespace gbn
