// kv.cuh -- the 8-bit cache format: device helpers shared by the cache
// writer and reader (kv_cache.cu) and the attention over it.
//
// A block of 32 elements has one scale byte b, the scale is 2^(b - 127); 255
// stands for NaN.  The writer uses 3 .. 249 and, for a block of zeros, 0; a
// caller's own cache may hold any byte, and all kernels take the same number.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace wide {

constexpr int kKvHD = 128;          // elements of a row
constexpr int kKvBlock = 32;        // elements per scale
constexpr int kKvMinExp = -124;     // smallest scale: keeps 2^-9 of it (e4m3's step) a bf16 number

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Scale byte of a block whose largest magnitude is `top` (bits of a
// non-negative fp32): the smallest exponent e >= kKvMinExp with
// top <= kMax * 2^e; 0 for a block of zeros, 255 for one that is not finite.
// top = 1.f * 2^p with kMax = 1.m * 2^q gives e = p - q, one more when the
// mantissa is above kMax's (448 = 1.75 * 2^8, 127 = 1.984375 * 2^6).
template <int KIND>
__device__ __forceinline__ uint32_t kv_scale_byte(uint32_t top)
{
    constexpr int kQ = KIND == WIDE_KV_E4M3 ? 8 : 6;
    constexpr uint32_t kMant = KIND == WIDE_KV_E4M3 ? 0x600000u : 0x7E0000u;
    if (top >= 0x7f800000u)
        return 255u;
    if (top == 0u)
        return 0u;
    const int e = (int)(top >> 23) - 127 - kQ + ((top & 0x7fffffu) > kMant ? 1 : 0);
    return (uint32_t)(max(e, kKvMinExp) + 127);
}

// 8 elements in the code of a block with scale byte b (0 and 255: zeros).
// x * 2^-e is exact (or far below half the smallest code), so each code is
// the correctly rounded one.
template <int KIND>
__device__ __forceinline__ uint2 kv_encode8(const float (&x)[8], uint32_t b)
{
    const float r = (b == 0u || b == 255u) ? 0.f : exp2i(127 - (int)b);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (KIND == WIDE_KV_E4M3) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                make_float2(x[4 * i] * r, x[4 * i + 1] * r), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(x[4 * i + 2] * r, x[4 * i + 3] * r), __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        } else {
            // 1.5 * 2^23 added: the sum's low byte is the product rounded to a whole
            // number (ties to even), with no conversion instruction
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = __float_as_uint(fmaf(x[4 * i + k], r, 12582912.f));
            w[i] = __byte_perm(__byte_perm(v[0], v[1], 0x0040), __byte_perm(v[2], v[3], 0x0040), 0x5410);
        }
    }
    return b == 255u ? make_uint2(0u, 0u) : make_uint2(w[0], w[1]);
}

// Multiplier of a block with scale byte b (2^-127 is not a normal number).
__device__ __forceinline__ float kv_scale(uint32_t b)
{
    return __uint_as_float(b == 255u ? 0x7fffffffu : max(b << 23, 0x00400000u));
}

// 4 codes (one word) as fp32 numbers times `scale`.
template <int KIND>
__device__ __forceinline__ void kv_decode4(uint32_t w, float scale, float (&f)[4])
{
    if constexpr (KIND == WIDE_KV_E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            f[2 * i] = v.x * scale;
            f[2 * i + 1] = v.y * scale;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = (float)(int)(int8_t)(w >> (8 * i)) * scale;
    }
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Multiplier that turns a code, moved into bf16 bits, into its value.  e4m3:
// the bits stand for value * 2^-120, so the multiplier is 2^(b - 127 + 120);
// above 2^127 (b > 134) the rest goes into a second one, kv_mult_high.  i8: it is
// the scale itself, 2^-127 not a normal number.
template <int KIND> __device__ __forceinline__ uint32_t kv_mult(uint32_t b)
{
    if (b == 255u)
        return 0x7fffu;
    return KIND == WIDE_KV_E4M3 ? min(b + 120u, 254u) << 7 : max(b << 7, 0x40u);
}
__device__ __forceinline__ uint32_t kv_mult_high(uint32_t b)
{
    return (b > 134u && b < 255u ? b - 7u : 127u) << 7;
}

// kv_mult of the scale bytes in the two halves of b.  i8: three instructions for
// both; 255 becomes an infinity, and inf * 0 + inf is NaN.
template <int KIND> __device__ __forceinline__ uint32_t kv_mult2(uint32_t b)
{
    if constexpr (KIND == WIDE_KV_E4M3) {
        return kv_mult<KIND>(b & 255u) | kv_mult<KIND>(b >> 16) << 16;
    } else {
        const uint32_t m = __vmaxu2(b << 7, 0x00400040u);
        uint32_t d;
        asm("fma.rn.bf16x2 %0, %1, %2, %1;" : "=r"(d) : "r"(m), "r"(0u));
        return d;
    }
}

// Two codes, in the bytes of t that the kind wants (e4m3: the high byte of
// each half; i8: the low byte; the other byte is ignored), as bf16 times mult.
// opaque: kv_opaque(kind), as a value that the compiler does not know.  i8: an
// and-or with two immediate operands is two instructions, with one and a
// register it is one.  e4m3: a left shift is a product in the other pipe.
__host__ __device__ constexpr uint32_t kv_opaque(int kind) { return kind == WIDE_KV_E4M3 ? 16u : 0x43004300u; }
template <int KIND> __device__ __forceinline__ uint32_t kv_pair(uint32_t t, uint32_t mult, uint32_t opaque)
{
    if constexpr (KIND == WIDE_KV_E4M3) {
        // sign, exponent and mantissa to bf16's places: s eeee mmm -> s 0000eeee mmm0000
        return mul_bf16x2(((t >> 4) & 0x07f007f0u) | (t & 0x80008000u), mult);
    } else {
        // 128 + (x & 127) as bf16, minus 128, or minus 256 if the sign bit is set
        const uint32_t u = (t & 0x007f007fu) | opaque, z = (t & 0x00800080u) | opaque;
        return mul_bf16x2(sub_bf16x2(u, z), mult);
    }
}

// The four codes of word x as bf16 times mult: bytes 0 and 2 in a, 1 and 3 in
// b.  Bytes two apart are in the two halves already, so there is no permute:
// five integer instructions a word.
template <int KIND>
__device__ __forceinline__ void kv_pairs_0213(uint32_t x, uint32_t mult, uint32_t opaque, uint32_t &a, uint32_t &b)
{
    if constexpr (KIND == WIDE_KV_E4M3) {
        const uint32_t y = x * opaque, z = y * opaque;    // x << 4, x << 8
        a = mul_bf16x2((y & 0x07f007f0u) | (z & 0x80008000u), mult);
        b = mul_bf16x2(((x >> 4) & 0x07f007f0u) | (x & 0x80008000u), mult);
    } else {
        a = kv_pair<KIND>(x, mult, opaque);
        b = kv_pair<KIND>(x >> 8, mult, opaque);
    }
}

}  // namespace wide
