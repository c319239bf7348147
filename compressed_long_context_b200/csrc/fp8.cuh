// fp8.cuh -- the 8-bit entry format and its tensor-core helpers.
//
// An 8-bit cache entry of one (row, KV head) is d e4m3 codes of the pooled key, dv of the pooled
// value and two e8m0 scales (bytes: key, value; byte u stands for 2^(u - 127)).  The scale of a
// vector is the smallest 2^e with max|x| <= 448 * 2^e, e clamped to [-64, 120]; its codes are x / 2^e
// rounded to the nearest e4m3 value (ties to even).  A power of two loses nothing against max|x| / 448:
// e4m3 is a floating format, so the relative step of a code does not depend on the scale, and both
// x / 2^e and code * 2^e are exact.  The step is 2^-3 of the power of two below |x| (half a step is at
// most 2^-4 of |x|) down to 2^-6 * 2^e, and 2^-9 * 2^e below; 2^-6 * 2^e is at most 2^-13.8 of max|x|.
// e4m3 has no infinity: a value that is not finite becomes the NaN code, and takes no part in the
// maximum.  At 2^120 codes end at 240, since 256 * 2^120 is more than bf16 and fp32 hold (bf16's largest
// value, 255 * 2^120, is 2^-4 of itself off then).  The clamp at 2^-64 bounds the sums of decode_quant.cuh, which carry 1 / scale.
#pragma once

#include "common.cuh"

namespace hca {

constexpr int kQMinExp = -64, kQMaxExp = 120;

// e8m0 byte of the scale for a largest magnitude `amax` (finite, >= 0).
__device__ __forceinline__ uint32_t q_scale_byte(float amax) {
    const uint32_t u = __float_as_uint(amax);
    // amax = f * 2^x, 1 <= f < 2; 448 = 1.75 * 2^8
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, kQMinExp), kQMaxExp);
    return (uint32_t)(e + 127);
}
// 2^(byte - 127) and its reciprocal
__device__ __forceinline__ float q_scale(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float q_inv_scale(uint32_t byte) {
    return __uint_as_float((uint32_t)max(254 - (int)byte, 0) << 23);
}

// |x| if finite, else 0 (what a vector's maximum is taken over)
__device__ __forceinline__ float q_mag(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;
}

// Two values to e4m3 / e5m2 codes (a in the low byte), nearest even.  The conversion saturates; values
// scaled by their own maximum stay inside the range.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t cvt_e5m2x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// Two e4m3 codes (low 16 bits of c) to fp32; every e4m3 value is an fp16 value.
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    float2 f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}

// Two values (at most 448 in magnitude, or NaN) as two e4m3 terms each: returns the codes of the values, sets those of what
// is left.  The difference is taken in fp16, which holds 11 bits of the value and the code exactly.
__device__ __forceinline__ uint32_t q_split(float a, float b, uint32_t& rest) {
    uint32_t out, r;
    asm("{\n\t.reg .b32 v, c, n;\n\t.reg .b16 h, l;\n\t"
        "cvt.rn.f16x2.f32 v, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 h, v;\n\t"
        "cvt.rn.f16x2.e4m3x2 c, h;\n\t"
        "sub.f16x2 n, v, c;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 l, n;\n\t"
        "cvt.u32.u16 %0, h;\n\tcvt.u32.u16 %1, l;\n\t}"
        : "=r"(out), "=r"(r) : "f"(a), "f"(b));
    rest = r;
    return out;
}

// A code for x * inv: NaN for a value that is not finite.  (x * inv is at most 448 in magnitude for
// every finite x that took part in the maximum.)
__device__ __forceinline__ float q_prep(float x, float inv) { return fabsf(x) < INFINITY ? x * inv : NAN; }

// Codes of entries' values, held where their value is finite in bf16.
constexpr float kQTop = 0x1.ep+127f;                    // 240 * 2^120
__device__ __forceinline__ float q_hold(float x, float inv) {
    return q_prep(fabsf(x) < INFINITY ? fminf(fmaxf(x, -kQTop), kQTop) : x, inv);
}
__device__ __forceinline__ uint32_t q_codes2(float a, float b, float inv) { return cvt_e4m3x2(q_hold(a, inv), q_hold(b, inv)); }
__device__ __forceinline__ uint32_t q_codes4(float4 x, float inv) {
    return q_codes2(x.x, x.y, inv) | q_codes2(x.z, x.w, inv) << 16;
}

// ------------------------------------------------------------------ tcgen05, kind::f8f6f4

enum : uint32_t { kFmtE4M3 = 0, kFmtE5M2 = 1 };

// Instruction descriptor: fp32 accumulate, A and B of the given 8-bit formats (K = 32 per MMA).
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, uint32_t afmt, uint32_t bfmt, int a_mn, int b_mn) {
    return (1u << 4) | (afmt << 7) | (bfmt << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// Descriptor of a 64-byte-swizzled operand (rows of 64 bytes, 8-row groups 512 bytes apart).
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)((lbo_bytes >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)((sbo_bytes >> 4) & 0x3FFF) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)4 << 61;
    return d;
}

// Byte offset of 16-byte chunk `c` (0..3) of row `r` in a 64-byte-swizzled tile.
__device__ __forceinline__ uint32_t sw64(uint32_t r, uint32_t c) { return r * 64u + (((c ^ (r >> 1)) & 3u) << 4); }

}  // namespace hca
