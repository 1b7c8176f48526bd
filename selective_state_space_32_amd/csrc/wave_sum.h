// Sums over the lanes of a wave by data-parallel primitives, without LDS.
#pragma once

#include <type_traits>

#include <hip/hip_runtime.h>

namespace ssm {

// Sum over the wave's lanes, in every lane (row shifts, then the two row broadcasts).
__device__ __forceinline__ float wave_sum(float v) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x111, 0xf, 0xf, false));  // row_shr:1
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x112, 0xf, 0xf, false));  // row_shr:2
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x114, 0xf, 0xf, false));  // row_shr:4
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x118, 0xf, 0xf, false));  // row_shr:8
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xa, 0xf, false));  // row_bcast:15
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xc, 0xf, false));  // row_bcast:31
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sum over LANES (8 to 64) neighbouring lanes of a wave, in each of them.
template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (LANES == 64) {
        return wave_sum(v);
    } else {
        auto dpp = [](float x, auto c) {
            return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), c.value, 0xf, 0xf, false));
        };
        v += dpp(v, std::integral_constant<int, 0xb1>{});    // quad_perm 1 0 3 2
        v += dpp(v, std::integral_constant<int, 0x4e>{});    // quad_perm 2 3 0 1
        v += dpp(v, std::integral_constant<int, 0x141>{});   // row_half_mirror: the other four of eight
        if constexpr (LANES >= 16) v += dpp(v, std::integral_constant<int, 0x140>{});   // row_mirror
        if constexpr (LANES >= 32) v += __shfl_xor(v, 16, 64);
        return v;
    }
}
}  // namespace ssm
