// mx.h -- rows in 8 bits (OCP Microscaling, MXFP8 with E4M3 elements): every 32
// consecutive elements of a row share one scale 2^(s - 127), s the byte of E8M0.
//
// The scale is the least power of two with amax <= 448 scale (amax the block's
// largest finite size, 448 the largest E4M3 number), so no element saturates;
// the other rule in use, 2^(floor(log2 amax) - 8), clips the eighth of each
// octave above 448 and saves nothing on the rest.  Elements are v / scale
// rounded to nearest even: off by at most 2^-4 of the value, or 2^-10 scale
// below the normal range (2^-6 scale).  A value that is not finite becomes the
// NaN code (E4M3 has no infinity) and leaves its block's scale alone.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace rssm {

constexpr int kMxBlock = 32;   // elements that share a scale

namespace {

// Type tag of an MX output in the kernels' output type parameter.
struct mx8 {};

// Bits of |v| when v is finite, else 0 (as integers they order as the sizes do).
__device__ __forceinline__ uint32_t mx_size(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}

// E8M0 byte of a block's amax (bits).  448 = 1.75 2^8: the exponent goes up by
// one where the mantissa is over 1.75, which the sum's carry does.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax) {
    const uint32_t e = (amax + 0x1FFFFFu) >> 23;
    return e > 8u ? e - 8u : 0u;
}

// 1 / scale; a normal number for every byte that mx_scale gives (0..247).
__device__ __forceinline__ float mx_inverse(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// Largest of four neighbouring lanes' numbers.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadSwap1, 0xF, 0xF, false));
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadRev, 0xF, 0xF, false));
}

// Four elements to codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t mx_codes(float a, float b, float c, float d, float inv) {
    const auto q = [inv](float v) {   // (products with a power of two are exact here, or round once below 2^-126)
        return (__float_as_uint(v) & 0x7FFFFFFFu) < 0x7F800000u ? v * inv : __builtin_nanf("");
    };
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(q(a), q(b), 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(q(c), q(d), r, true);
    return (uint32_t)r;
}

}  // namespace
}  // namespace rssm
