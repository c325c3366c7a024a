// elem.hpp -- element types of the operators for rounded layers: loads of 8
// values as fp32, and conversions back.
#pragma once

#include "common.hpp"

namespace bakron {

// Row strides are bounded so that 64-bit byte offsets cannot overflow.
constexpr int64_t MAX_LD = int64_t(1) << 32;

inline int64_t elem_size(int32_t type) { return type == BAKRON_T_F32 ? 4 : 2; }

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float x) {
    const __bf16 h = (__bf16)x;  // round to nearest, ties to even
    uint16_t b;
    __builtin_memcpy(&b, &h, 2);
    return b;
}

__device__ __forceinline__ uint16_t f32_to_f16(float x) {
    const _Float16 h = (_Float16)x;
    uint16_t b;
    __builtin_memcpy(&b, &h, 2);
    return b;
}

__device__ __forceinline__ float f16_to_f32(uint16_t b) {
    _Float16 h;
    __builtin_memcpy(&h, &b, 2);
    return (float)h;
}

template <int T>
__device__ __forceinline__ float load1(const char *base, int64_t i) {
    if constexpr (T == BAKRON_T_F32) return reinterpret_cast<const float *>(base)[i];
    const uint16_t b = reinterpret_cast<const uint16_t *>(base)[i];
    return T == BAKRON_T_BF16 ? bf16_to_f32(b) : f16_to_f32(b);
}

template <int T>
__device__ __forceinline__ void unpack8(const uint32_t *w, float *x) {
    if constexpr (T == BAKRON_T_F32) {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = __uint_as_float(w[q]);
    } else if constexpr (T == BAKRON_T_BF16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[2 * q] = __uint_as_float(w[q] << 16);
            x[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[2 * q] = f16_to_f32((uint16_t)w[q]);
            x[2 * q + 1] = f16_to_f32((uint16_t)(w[q] >> 16));
        }
    }
}

// x[0..7] = elements i .. i + 7 of `base` as fp32; those from `left` on are 0
// and not read.  The address needs the alignment of one element only.
template <int T>
__device__ __forceinline__ void load8(const char *base, int64_t i, int64_t left, float *x) {
    constexpr int ES = T == BAKRON_T_F32 ? 4 : 2;
    if (left >= 8) {
        uint32_t w[2 * ES];
        __builtin_memcpy(w, base + i * ES, 8 * ES);
        unpack8<T>(w, x);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = q < left ? load1<T>(base, i + q) : 0.0f;
    }
}

// Bit pattern of 2 values in a 16-bit type, low half first.
template <int T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef float floatx2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const floatx2 v = {a, b};
    if constexpr (T == BAKRON_T_BF16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

template <int T>
__device__ __forceinline__ void store1(char *base, int64_t i, float x) {
    if constexpr (T == BAKRON_T_F32)
        reinterpret_cast<float *>(base)[i] = x;
    else
        reinterpret_cast<uint16_t *>(base)[i] = T == BAKRON_T_BF16 ? f32_to_bf16(x) : f32_to_f16(x);
}

// elements i .. i + 7 of `base` = x[0..7] rounded to the type; from `left` on nothing is written
template <int T>
__device__ __forceinline__ void store8(char *base, int64_t i, int64_t left, const float *x) {
    constexpr int ES = T == BAKRON_T_F32 ? 4 : 2;
    if (left >= 8) {
        uint32_t w[2 * ES];
        if constexpr (T == BAKRON_T_F32) {
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] = __float_as_uint(x[q]);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = pack2<T>(x[2 * q], x[2 * q + 1]);
        }
        __builtin_memcpy(base + i * ES, w, 8 * ES);
    } else {
        for (int q = 0; q < left; ++q) store1<T>(base, i + q, x[q]);
    }
}

}  // namespace bakron
