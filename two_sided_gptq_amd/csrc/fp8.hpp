// fp8.hpp -- conversion of blocks of values to 8-bit floating point (e4m3: 4 exponent
// bits, 3 mantissa bits, largest value 448), shared by the calls that quantise.
#pragma once

#include "common.hpp"

namespace bakron {

constexpr float FP8_MAX = 448.0f;
// A block's largest magnitude is taken as at least 2^-100, so that 448 / amax
// stays finite; a block of zeros gets the scale 1.
constexpr float AMAX_FLOOR = 0x1p-100f;

// The largest magnitude travels as its bit pattern: as unsigned integers,
// magnitudes compare in order and a NaN is above them all.
__device__ __forceinline__ void block_scale(uint32_t amax_bits, float &scale, float &inv, bool &bad) {
    bad = amax_bits >= 0x7f800000u;
    float amax = __uint_as_float(amax_bits);
    amax = amax_bits == 0 ? FP8_MAX : fmaxf(amax, AMAX_FLOOR);
    scale = bad ? __uint_as_float(0x7fc00000u) : amax / FP8_MAX;
    inv = FP8_MAX / amax;
}

// 8 values to 8 codes.  x inv can round to just over 448, hence the clamp; the
// conversion rounds to nearest, ties to even.  A bad block is all NaN codes.
__device__ __forceinline__ uint2 encode8(const float *x, float inv, bool bad) {
    if (bad) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) c[q] = fminf(fmaxf(x[4 * h + q] * inv, -FP8_MAX), FP8_MAX);
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
        w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], v, true);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store8(uint8_t *dst, uint2 v, int count) {
    if (count >= 8) {
        __builtin_memcpy(dst, &v, 8);
    } else {
        const uint64_t u = ((uint64_t)v.y << 32) | v.x;
        for (int q = 0; q < count; ++q) dst[q] = (uint8_t)(u >> (8 * q));
    }
}

// Maximum over the 16 lanes of a DPP row, in every lane.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));  // row_ror:8
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
    return v;
}

}  // namespace bakron
