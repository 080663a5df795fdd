// Values of 8 bits under a shared scale: e4m3 codes c and a scale byte b, a
// value being c * 2^(b - 127). The scale of a set of values is the smallest
// 2^e, e >= -127, under which none saturates: with a the largest finite
// magnitude, a <= 464 * 2^e (464 is the largest number that rounds to e4m3's
// 448). Because that is where the rounding of a changes its code's exponent, the
// codes themselves tell the same e again.
//
// Coding rounds once, to nearest even: by at most 2^-4 of a value of
// 2^-6 * 2^e or more (a power of two cancels, so the scale does not matter),
// else by at most 2^-10 * 2^e, which is below 2^-17 of a. What is not finite
// becomes NaN and does not count in a.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "tf_internal.cuh"

namespace tf {

constexpr int kScaleBias = 127;

// |x| as bits, 0 for what is not finite: the largest of these gives the scale.
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
    return u < 0x7F800000u ? u : 0u;
}
// The exponent e of the largest finite magnitude, given as bits. With a = 1.f * 2^(x - 127):
// 464 = 1.8125 * 2^8, so e = x - 135, or one more where 1.f is above 1.8125.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
    const int e = int(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x680000u ? 1 : 0);
    return e > -kScaleBias ? e : -kScaleBias;
}
// 2^-e for an exponent that scale_exponent returned (-127..120): a normal number.
__device__ __forceinline__ float scale_inverse(int e) { return __uint_as_float(uint32_t(127 - e) << 23); }
// 2^(b - 127) of a scale byte, 2^-127 as the subnormal it is.
__device__ __forceinline__ float scale_value(uint32_t b) {
    return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// Codes of two numbers (a low, b high) that are already divided by the scale.
__device__ __forceinline__ uint16_t e4m3_pair(float a, float b) {
    // an infinity would become the largest code
    a = fabsf(a) <= 464.f ? a : __uint_as_float(0x7FC00000u);
    b = fabsf(b) <= 464.f ? b : __uint_as_float(0x7FC00000u);
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
    return d;
}
// The same where neither is an infinity.
__device__ __forceinline__ uint32_t e4m3_finite(float a, float b) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
    return d;
}
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
    return uint32_t(e4m3_pair(a, b)) | uint32_t(e4m3_pair(c, d)) << 16;
}
// Two codes (in a register's low or high half) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3_to_h2(uint16_t x) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(x));
    return d;
}
__device__ __forceinline__ uint32_t e4m3_low(uint32_t w) { return e4m3_to_h2(uint16_t(w)); }
__device__ __forceinline__ uint32_t e4m3_high(uint32_t w) { return e4m3_to_h2(uint16_t(w >> 16)); }
__device__ __forceinline__ float2 h2_to_f2(uint32_t h) { return __half22float2(*reinterpret_cast<__half2*>(&h)); }

// ---- the launches of tables of scaled pools --------------------------------

// attn_scaled.cu: the attention partials (the records and merges of attn.cu), and
// the kernels' attributes.
int launch_attn_scaled(const SegTable& t, int layer, const uint16_t* q, float* po, float2* pml, cudaStream_t stream,
                       uint16_t* out, int full);
int attn_scaled_prepare();
// attn_scaled_tc.cu: the tensor-core part of them, items [n_items_mma, n_items);
// grid_cap 0: two CTAs an SM.
int launch_attn_scaled_tc(const SegTable& t, int layer, const uint16_t* q, float* po, float2* pml, cudaStream_t stream,
                          uint16_t* out, int full, int grid_cap = 0);
int attn_scaled_tc_prepare();

// qk_scaled.cu: the append with the queries' norm and rotation (tf_qk_rows).
struct Turns {
    uint64_t f[TF_D / 2];   // f_j as a fraction of a turn, 2^64 = one turn
};
struct QkvRows {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride;
};
int launch_qk_scaled(const SegTable& t, int layer, const QkvRows& in, const uint16_t* q_norm, const uint16_t* k_norm,
                     float eps, const Turns& turns, uint16_t* q_out, cudaStream_t stream);

}  // namespace tf
