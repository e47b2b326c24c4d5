// Quantizing blocks of values to E4M3 with a power-of-two scale, in registers
// (gfx950).
//
// t = the smallest integer with 448 * 2^t >= the block's largest magnitude (0 for
// zeros), at least -127; the E8M0 byte is t + 127, the codes are E4M3(v / 2^t) to
// nearest even.  The scaled conversions v_cvt_scalef32_pk_fp8_* do this for two
// values at a time, with the scale as an operand and without rounding before:
// exact for every bf16 and f16 pattern at scales from 2^-127 to 2^120 (compared
// exhaustively with a multiplication and v_cvt_pk_fp8_f32).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg_device.h"

namespace gfg {
namespace {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Eight neighbouring elements as they lie in memory.  `w2`: the second four of 32 bits.
template <typename T> struct Eight {
    u32x4 w;
    __device__ __forceinline__ float at(int i) const {
        const uint16_t h = uint16_t(w[i >> 1] >> (16 * (i & 1)));
        return float(__builtin_bit_cast(T, h));
    }
};
template <> struct Eight<float> {
    u32x4 w, w2;
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(i < 4 ? w[i & 3] : w2[i & 3]); }
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
    Eight<T> e;
    e.w = reinterpret_cast<const u32x4*>(p)[0];
    if constexpr (sizeof(T) == 4) e.w2 = reinterpret_cast<const u32x4*>(p)[1];
    return e;
}
// by a buffer load: zeros outside the window
template <typename T>
__device__ __forceinline__ Eight<T> load8(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    Eight<T> e;
    e.w = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
    if constexpr (sizeof(T) == 4) e.w2 = __builtin_amdgcn_raw_buffer_load_b128(r, at + 16, 0, 0);
    return e;
}

// Largest magnitudes.  Of 32 bits: the magnitude's bits, whose integer order is
// the magnitudes', with infinities and NaN above every finite value.  Of 16 bits:
// two of them in a word, each with the same order.
template <typename T>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return max(a, b);
    else return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
template <typename T>
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return w & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu); }
template <typename T>
__device__ __forceinline__ uint32_t largest(const Eight<T>& e) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = larger<T>(m, magnitudes<T>(e.w[i]));
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = larger<T>(m, magnitudes<T>(e.w2[i]));
    }
    return m;
}
// One magnitude's fp32 bits: of the half h of a word, or of the larger half.
template <typename T>
__device__ __forceinline__ uint32_t as_f32(uint32_t m, int h) {
    if constexpr (sizeof(T) == 4) {
        return m;
    } else {
        const uint16_t v = uint16_t(h ? m >> 16 : m);
        return __float_as_uint(float(__builtin_bit_cast(T, v)));
    }
}
template <typename T>
__device__ __forceinline__ uint32_t as_f32(uint32_t m) {
    if constexpr (sizeof(T) == 4) return m;
    else return as_f32<T>(max(m & 0xFFFFu, m >> 16), 0);
}

// A block's E8M0 byte from its largest magnitude's fp32 bits.  448 = 1.75 * 2^8 and
// max = 1.f * 2^e give t = e - 8, one more where 1.f > 1.75, that is where adding
// 0x1FFFFF to the mantissa bits 0x600000 and above carries.  (A subnormal maximum
// would have t below -127.)  An infinity or a NaN: 255, E8M0's NaN.
__device__ __forceinline__ uint32_t scale_byte_of(uint32_t ab) {
    const int b = max(int((ab + 0x1FFFFFu) >> 23) - 8, 0);
    return ab == 0 ? 127u : ab >= 0x7F800000u ? 255u : uint32_t(b);
}
// The scale 2^(byte - 127) as the conversions take it.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }
// All ones where there is none: the codes of NaN go in.
__device__ __forceinline__ uint32_t none_of(uint32_t byte) { return byte == 255u ? 0xFFFFFFFFu : 0u; }
__device__ __forceinline__ uint32_t or_nan(uint32_t codes, uint32_t none) { return (codes & ~none) | (0x7F7F7F7Fu & none); }

// Two codes of a word of two 16-bit values, or of two 32-bit values, into a half of `old`.
template <typename T, bool HI>
__device__ __forceinline__ uint32_t two(uint32_t old, uint32_t w, float scale) {
    if constexpr (__is_same(T, __bf16))
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(__builtin_bit_cast(i16x2, old), __builtin_bit_cast(bf16x2, w), scale, HI));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(__builtin_bit_cast(i16x2, old), __builtin_bit_cast(f16x2, w), scale, HI));
}
template <bool HI>
__device__ __forceinline__ uint32_t two(uint32_t old, float a, float b, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(__builtin_bit_cast(i16x2, old), a, b, scale, HI));
}
__device__ __forceinline__ uint32_t four(float a, float b, float c, float d, float scale) {
    return two<true>(two<false>(0u, a, b, scale), c, d, scale);
}
template <typename T>
__device__ __forceinline__ u32x2 encode(const Eight<T>& e, uint32_t byte) {
    const float scale = scale_of(byte);
    const uint32_t none = none_of(byte);
    u32x2 o;
    if constexpr (sizeof(T) == 4) {
        o[0] = four(e.at(0), e.at(1), e.at(2), e.at(3), scale);
        o[1] = four(e.at(4), e.at(5), e.at(6), e.at(7), scale);
    } else {
        o[0] = two<T, true>(two<T, false>(0u, e.w[0], scale), e.w[1], scale);
        o[1] = two<T, true>(two<T, false>(0u, e.w[2], scale), e.w[3], scale);
    }
    return u32x2{or_nan(o[0], none), or_nan(o[1], none)};
}

}  // namespace
}  // namespace gfg
