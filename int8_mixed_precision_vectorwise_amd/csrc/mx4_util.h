// Device helpers of the microscaled 4-bit kernels (gfx950 only).
#pragma once

#include "common.h"
#include "mx4.h"

namespace i8mp {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef _Float16 hh2 __attribute__((ext_vector_type(2)));
typedef __bf16 bb2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));

// the scale's byte from the bits of the largest magnitude
template <bool kBf16>
__device__ inline uint32_t scale_byte(uint32_t top) {
    // fp16's subnormal numbers are normal in fp32; bfloat16's get the least scale
    const uint32_t bits = kBf16 ? top << 16 : __float_as_uint(h2f((half_bits)top));
    const uint32_t e = bits >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^(byte - 127); 255 gives a NaN
__device__ inline float scale_value(uint32_t byte) {
    return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}

__device__ inline us2 mags(uint32_t w) { return __builtin_bit_cast(us2, w & 0x7fff7fffu); }

// byte kSel of `old` := codes of a pair of 16-bit values
template <bool kBf16, int kSel>
__device__ inline uint32_t encode2(uint32_t old, uint32_t w, float scale) {
    if constexpr (kBf16) return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bb2, w), scale, kSel);
    else return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(hh2, w), scale, kSel);
}
template <bool kBf16>
__device__ inline uint32_t encode8(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, float scale) {
    uint32_t c = encode2<kBf16, 0>(0u, w0, scale);
    c = encode2<kBf16, 1>(c, w1, scale);
    c = encode2<kBf16, 2>(c, w2, scale);
    return encode2<kBf16, 3>(c, w3, scale);
}

// ---- operands and buffers -------------------------------------------------------

constexpr int kOut = (int)0x80000000;    // makes a buffer offset leave every range: reads zeros

__device__ inline __amdgpu_buffer_rsrc_t range_of(const void* base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

__device__ inline v8i operand(const v4i& x) { return __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1); }

__device__ inline float widen(const void* p, int64_t i, int dtype) {
    if (dtype == I8MP_DTYPE_F32) return static_cast<const float*>(p)[i];
    const half_bits h = static_cast<const half_bits*>(p)[i];
    return dtype == I8MP_DTYPE_BF16 ? __uint_as_float((uint32_t)h << 16) : h2f(h);
}
template <int kType>
__device__ inline uint32_t narrow2(float x, float y) {
    if constexpr (kType == I8MP_DTYPE_BF16)
        return __builtin_bit_cast(half_bits, (__bf16)x) | (uint32_t)__builtin_bit_cast(half_bits, (__bf16)y) << 16;
    else return f2h(x) | (uint32_t)f2h(y) << 16;
}

}  // namespace i8mp
