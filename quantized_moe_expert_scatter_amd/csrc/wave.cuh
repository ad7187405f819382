// wave.cuh -- reductions over a 64-lane wavefront and element conversions,
// shared by the router, combine-gradient and adapter kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace moe {

constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;      // moe_dtype

template <int DT> struct Elem { using T = float; };
template <> struct Elem<kBF16> { using T = uint16_t; };
template <> struct Elem<kF16> { using T = uint16_t; };

template <int DT>
__device__ __forceinline__ float to_float(typename Elem<DT>::T e) {
    if constexpr (DT == kF32) return e;
    else if constexpr (DT == kBF16) return __uint_as_float(uint32_t(e) << 16);
    else return float(__builtin_bit_cast(_Float16, e));
}

// Rounded to nearest even; a NaN stays one.
template <int DT>
__device__ __forceinline__ typename Elem<DT>::T from_float(float f) {
    if constexpr (DT == kF32) return f;
    else if constexpr (DT == kBF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
    else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}

// One step of a reduction through the data-parallel primitives: the value a
// lane CTRL away in its row (or the row broadcasts 0x142, 0x143), 0 where
// there is none, so 0 must be the operation's identity.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xf, true));
}

// Largest of the wave's values, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp0<0x111, 0xf>(v));
    v = max(v, dpp0<0x112, 0xf>(v));
    v = max(v, dpp0<0x114, 0xf>(v));
    v = max(v, dpp0<0x118, 0xf>(v));
    v = max(v, dpp0<0x142, 0xa>(v));
    v = max(v, dpp0<0x143, 0xc>(v));
    return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

// Sum over the wave in a fixed order, in every lane.
__device__ __forceinline__ float wave_sum(float f) {
    auto step = [](float x, uint32_t y) { return x + __uint_as_float(y); };
    f = step(f, dpp0<0x111, 0xf>(__float_as_uint(f)));
    f = step(f, dpp0<0x112, 0xf>(__float_as_uint(f)));
    f = step(f, dpp0<0x114, 0xf>(__float_as_uint(f)));
    f = step(f, dpp0<0x118, 0xf>(__float_as_uint(f)));
    f = step(f, dpp0<0x142, 0xa>(__float_as_uint(f)));
    f = step(f, dpp0<0x143, 0xc>(__float_as_uint(f)));
    return __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(f)), 63)));
}

}  // namespace moe
