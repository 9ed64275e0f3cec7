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
// its largest magnitude.  The definition's float64 quotients, rounded to fp32,
// are the fp32 quotients here: where hi - lo is exact in fp32 (checked), a
// quotient of a 24-bit number by 15, or by a scale of 8 bits, is at least
// 2^-33 of itself away from the middle of two fp32 numbers unless it is that
// middle, so that rounding it to 53 bits in between changes nothing.
__device__ __forceinline__ uint32_t kv4_word(float lo, float hi, uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 0x7fc0u;   // NaN or an infinity: scale NaN, offset 0
    float r = hi - lo;
    const float t = r - hi;                         // the difference's rounding error, exactly (two-sum)
    const float err = (hi - (r - t)) + (-lo - t);
    if (err == 0.f) r = __fdiv_rn(r, 15.f);
    else r = __double2float_rn(((double)hi - (double)lo) / 15.0);   // (also where r or err overflow)
    const bf16 s = __float2bfloat16_rn(fmaxf(r, __uint_as_float(amax_bits) * 0.0009765625f));
    const float sf = __bfloat162float(s);
    if (!(sf > 0.f)) return 0u;
    const f16 o = __float2half_rn(__fdiv_rn(lo, sf));
    return (uint32_t)__bfloat16_as_ushort(s) | ((uint32_t)__half_as_ushort(o) << 16);
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The codes of four values of a group with that parameter word, the first in
// the lowest four bits.  t = x / scale - off is taken as one fp32 multiply-add
// with an approximate reciprocal (within 2^-23 of itself): off by at most
// |x / scale| 2^-23 + |t| 2^-24 <= (|off| + 17) 2^-22 + 2^-19, so its rounding
// to an integer is the definition's unless t lies that close to a half; there,
// and where the reciprocal overflows, the float64 quotient decides.  t is at
// least -1/2 (offset's rounding) and at most 16 (scale's and offset's).
__device__ __forceinline__ uint32_t kv4_codes(const float (&x)[4], uint32_t word) {
    constexpr float M = 12582912.f;   // 1.5 2^23: adding it rounds to an integer, half to even
    const float scale = kv4_scale(word), off = kv4_offset(word);
    if (!(scale > 0.f)) return 0u;
    const float inv = rcp_approx(scale);
    const float lim = inv < 3e38f ? 0.5f - ((fabsf(off) + 17.f) * 2.4e-7f + 2e-6f) : -1.f;
    float r[4], far = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float t = fminf(fmaf(x[i], inv, -off), 15.f);
        r[i] = (t + M) - M;
        far = fmaxf(far, fabsf(t - r[i]));
    }
    if (!(far < lim)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = (float)fmin(fmax(rint((double)x[i] / (double)scale - (double)off), 0.0), 15.0);
    }
    // exact: at most 65535
    return (uint32_t)fmaf(r[3], 4096.f, fmaf(r[2], 256.f, fmaf(r[1], 16.f, r[0])));
}

}  // namespace la
