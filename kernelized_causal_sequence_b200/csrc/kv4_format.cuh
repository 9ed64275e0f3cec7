// kv4_format.cuh — the 4-bit cache rows (layout and quantisation: linattn.h,
// la_kv4_cache).
#pragma once
#include "common.cuh"

namespace la {

constexpr int kKv4Group = 32;     // channels that share a scale and an offset

__device__ __forceinline__ float kv4_scale(uint32_t word) { return __uint_as_float(word << 16); }
__device__ __forceinline__ float kv4_offset(uint32_t word) {
    return __half2float(__ushort_as_half((unsigned short)(word >> 16)));
}

// Scale and offset word of a group from its minimum, maximum and the bits of
// its largest magnitude.  float64, as the definition has it; a conversion to
// 16 bits goes through fp32.
__device__ __forceinline__ uint32_t kv4_word(float lo, float hi, uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 0x7fc0u;   // NaN or an infinity: scale NaN, offset 0
    const double r = ((double)hi - (double)lo) / 15.0;
    const double a = (double)__uint_as_float(amax_bits) / 1024.0;
    const bf16 s = __float2bfloat16_rn(__double2float_rn(r > a ? r : a));
    const float sf = __bfloat162float(s);
    if (!(sf > 0.f)) return 0u;
    const f16 o = __float2half_rn(__double2float_rn((double)lo / (double)sf));
    return (uint32_t)__bfloat16_as_ushort(s) | ((uint32_t)__half_as_ushort(o) << 16);
}

// The code of x in a group of that scale and offset; inv = 1 / scale in fp32.
// t = x inv - off in fp32 is within |x inv| 2^-22 + 2^-19 of the exact value
// (two roundings of the product and one of the difference, |t| < 32), so its
// rounding to an integer is the definition's unless t lies that close to a
// half; there the float64 quotient decides.
__device__ __forceinline__ uint32_t kv4_code(float x, float scale, float inv, float off) {
    if (!(scale > 0.f)) return 0u;
    const float y = x * inv, t = y - off, r = rintf(t);
    if (fabsf(t - r) < 0.5f - (fabsf(y) * 2.4e-7f + 2e-6f)) return (uint32_t)fminf(fmaxf(r, 0.f), 15.f);
    const double e = rint((double)x / (double)scale - (double)off);
    return (uint32_t)fmin(fmax(e, 0.0), 15.0);
}

}  // namespace la
