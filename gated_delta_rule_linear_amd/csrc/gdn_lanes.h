// Sums and maxima over the lanes of a wave without LDS: lanes 8, 4, 2, 1 apart by
// rotations within rows of 16, lanes 16 and 32 apart by row exchanges.  Every
// lane receives the result.
#pragma once

#include "gdn_device.h"

namespace gdn {

struct Sum {
    __device__ __forceinline__ static float of(float a, float b) { return a + b; }
};
struct Max {
    __device__ __forceinline__ static float of(float a, float b) { return fmaxf(a, b); }
};

template <int N>
__device__ __forceinline__ float rotated(float x) {  // within rows of 16 lanes
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x120 + N, 0xf, 0xf, false));
}
// Combines the lanes FROM, 2 FROM, ... TO apart (powers of two).
template <typename OP, int FROM = 1, int TO = 32>
__device__ __forceinline__ float across(float x) {
    if constexpr (FROM <= 1 && 1 <= TO) x = OP::of(x, rotated<1>(x));
    if constexpr (FROM <= 2 && 2 <= TO) x = OP::of(x, rotated<2>(x));
    if constexpr (FROM <= 4 && 4 <= TO) x = OP::of(x, rotated<4>(x));
    if constexpr (FROM <= 8 && 8 <= TO) x = OP::of(x, rotated<8>(x));
    if constexpr (FROM <= 16 && 16 <= TO) {
        const uint32_t u = __float_as_uint(x);
        const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        x = OP::of(__uint_as_float(p[0]), __uint_as_float(p[1]));
    }
    if constexpr (FROM <= 32 && 32 <= TO) {
        const uint32_t u = __float_as_uint(x);
        const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        x = OP::of(__uint_as_float(p[0]), __uint_as_float(p[1]));
    }
    return x;
}

}  // namespace gdn
