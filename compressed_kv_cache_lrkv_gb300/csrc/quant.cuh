// quant.cuh -- device helpers for the bytes of quantised rows.
#pragma once

#include "lrkv_internal.cuh"

namespace lrkv {

// Values q_i 2^k of two bytes (b0, b1 of [b0, 0, b1, 0]) as bf16, s2 = (2^k, 2^k): with the low seven
// bits in its mantissa bf16 holds 128 + u mod 128, from which 256 or, where the byte's top bit is
// set, 128 is taken; both steps and the product are exact.
__device__ __forceinline__ uint32_t bytes_bf16(uint32_t v, __nv_bfloat162 s2) {
    const uint32_t lo = (v & 0x007f007fu) | 0x43004300u, hi = (v & 0x00800080u) ^ 0x43804380u;
    const __nv_bfloat162 r = __hmul2(
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo), *reinterpret_cast<const __nv_bfloat162*>(&hi)), s2);
    return *reinterpret_cast<const uint32_t*>(&r);
}

// A block's scale twice in bf16: 2^(e - 127); NaN for byte 255, zero for 0 (a cleared row).
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t e) { return e == 255 ? 0x7fc07fc0u : e * 0x00800080u; }

}  // namespace lrkv
