// What the recurrence's kernels share: the decay of a log-decay, and four
// neighbouring channels.
#pragma once

#include "gdn_device.h"

namespace gdn {

__device__ __forceinline__ float decay(float g) { return __builtin_amdgcn_exp2f(1.4426950408889634f * g); }
// 1 - e^g without the difference's loss near g = 0: there by the exponential's
// series, whose next term is below 2^-23 of the sum; on the other side the decay's
// step of 2^-24 is below 2^-21 of the difference.
__device__ __forceinline__ float one_minus_decay(float g, float a) {
    float p = __builtin_fmaf(g, 1.f / 120.f, 1.f / 24.f);
    p = __builtin_fmaf(g, p, 1.f / 6.f);
    p = __builtin_fmaf(g, p, 0.5f);
    p = __builtin_fmaf(g, p, 1.f);
    p *= -g;
    asm("" : "+v"(p));  // (no branch around it: both sides are a few operations)
    return g > -0.15f ? p : 1.f - a;
}

// Four neighbouring values as they are in memory.
template <typename T>
struct Four;
template <>
struct Four<float> {
    typedef floatx4 raw;
    floatx4 v;
    __device__ __forceinline__ floatx4 f() const { return v; }
    __device__ __forceinline__ static floatx4 of(floatx4 x) { return x; }
};
template <>
struct Four<bf16> {
    typedef bf16x4 raw;
    bf16x4 v;
    __device__ __forceinline__ floatx4 f() const { return {(float)v[0], (float)v[1], (float)v[2], (float)v[3]}; }
    __device__ __forceinline__ static bf16x4 of(floatx4 x) { return {(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]}; }
};

}  // namespace gdn
