// rope.cuh -- rotary angles shared by the rotation kernel (rope.cu) and the
// cache writer (kv_cache.cu).
//
// The host computes the call's frequencies in double, as turns (radians over
// 2 pi) per position, and passes them as a kernel parameter: at most 128
// doubles, read through the constant bank.  A kernel then needs one double
// product and one rounding per angle: pos * turns, minus its nearest
// integer, is the angle within half a turn, whose cosine and sine are taken in
// fp32 (cospi / sinpi of twice that).  They are off by at most 4 * 2^-24 (the
// rounded argument, the functions, the amplitude) and, for an angle of x radians
// before the reduction, 8 * 2^-53 * |x| (the frequency's two powers and three
// roundings, the product's; the ramp's g makes it 16).  So they are as good as
// fp32 holds them up to 2^26 radians: position 2^26 where frequencies are at most
// 1 (theta >= 1, factor >= 1).  Position 2^31 adds 2^-19, a factor below 1 or a
// theta below 1 makes angles, and that error, larger.
#pragma once

#include "common.cuh"

namespace wide {

constexpr int kRopeMaxPairs = 128;

struct RopeTable {
    double turns[kRopeMaxPairs];   // of pair i per position
    float amplitude;
};

// Fills *t; false if the configuration is invalid (WIDE_EINVAL).
bool rope_table(const wide_rope_config *c, RopeTable *t);

// (A cos, A sin) of `pos` * turns.
__device__ __forceinline__ float2 rope_cos_sin(double turns, int32_t pos, float amplitude)
{
    const double a = (double)pos * turns;
    const float f = (float)(2.0 * (a - rint(a)));   // half turns in [-1, 1]
    float s, c;
    sincospif(f, &s, &c);
    return make_float2(c * amplitude, s * amplitude);
}

// Rotates the pair (a, b).  The product that is not fused is rounded by
// itself in every kernel, so all of them give the same bits.
__device__ __forceinline__ void rope_pair(float &a, float &b, float2 w)
{
    const float ra = fmaf(a, w.x, -__fmul_rn(b, w.y));
    b = fmaf(b, w.x, __fmul_rn(a, w.y));
    a = ra;
}

}  // namespace wide
