// The 8-bit format of the paged cache: e4m3 codes with a power-of-two scale.
#pragma once

#include "gdn_device.h"

namespace gdn {

typedef uint32_t uintx2 __attribute__((ext_vector_type(2)));
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));

constexpr int kMinScaleExponent = -100;

// The smallest power of two s >= 2^-100 with amax / s <= 448 = 1.75 * 2^8, from
// the bits of amax (finite, >= 0): one more than the exponent difference where
// the significand is above 1.75.
__device__ __forceinline__ float e4m3_scale(float amax) {
    const uint32_t b = __float_as_uint(amax);
    int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < kMinScaleExponent ? kMinScaleExponent : e;  // zero and subnormals too
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// |x| if it is finite, else 0.
__device__ __forceinline__ float finite_abs(float x) {
    const float y = fabsf(x);
    return y < __builtin_inff() ? y : 0.f;
}
// Inf becomes NaN, which has a code; the conversion itself would clamp it.
__device__ __forceinline__ float finite_or_nan(float x) {
    return fabsf(x) < __builtin_inff() ? x : __builtin_nanf("");
}
// Four values to four codes, round to nearest even.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
// The codes of a word times a power-of-two factor, rounded again.
__device__ __forceinline__ uint32_t e4m3_rescaled(uint32_t w, float f) {
    const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return to_e4m3(lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f);
}
// Two codes (the low or the high half of a word) as bf16 times a power of two,
// exactly (the result's exponent range is that of fp32).
template <bool HI>
__device__ __forceinline__ bf16x2 e4m3_to_bf16(uint32_t w, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, scale, HI);
}
__device__ __forceinline__ bf16x8 e4m3_to_bf16x8(uint32_t a, uint32_t b, float scale = 1.f) {
    const bf16x2 x = e4m3_to_bf16<false>(a, scale), y = e4m3_to_bf16<true>(a, scale), z = e4m3_to_bf16<false>(b, scale),
                 w = e4m3_to_bf16<true>(b, scale);
    return bf16x8{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
}
// Whether one of 16 codes is NaN (0x7f or 0xff).
__device__ __forceinline__ bool has_nan_code(uintx4 x) {
    uint32_t hit = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) hit |= ((x[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    return hit != 0;
}
// 0 in the place of NaN codes; in `ones` the code of 1 there and 0 elsewhere.
__device__ __forceinline__ void split_nan(uintx4& x, uintx4& ones) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t hit = (((x[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
        x[i] &= ~(hit * 0xffu);
        ones[i] = hit * 0x38u;
    }
}
// The first `count` of 16 codes (any number), 0 for the others.
__device__ __forceinline__ void keep_codes(uintx4& x, int64_t count) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int64_t left = count - 4 * w;
        x[w] &= left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * (int)left)) - 1u;
    }
}

}  // namespace gdn
