// mxfp4_encode.cuh -- MXFP4 block arithmetic shared by the quantizer and the linear layer's fused
// activation quantize, so that both produce identical codes and scales.
//
// MXFP4 (OCP Microscaling Formats, E2M1 elements): 32 values share one E8M0 byte b, 2^(b - 127).
// With E the biased fp32 exponent field of the block's largest magnitude m = 1.f * 2^(E - 127):
//   floor rule  2^(floor(log2 m) - 2): b = E - 2 (values in (6, 8) * 2^(b - 127) saturate);
//   ceil rule   the smallest power of two with m <= 6 * 2^(b - 127), 6 = 1.5 * 2^2: b = E - 2, one
//               more where 1.f > 1.5;
// both clamped at 0. (E = 0, subnormal m or a block of zeros, gives 0.) The largest b is 253, so
// 2^(127 - b), exponent field 254 - b >= 1, is a normal fp32. x * 2^(127 - b) is exact unless it
// is below 2^-126, where the code is 0 either way: codes are the round-to-nearest-even E2M1 of
// the exact quotient, saturating at 6, sign kept. A block that holds a NaN or an infinity gets
// b = 255 (NaN) and zero codes.
#pragma once
#include <cstdint>

#include "sm100_ptx.cuh"

namespace nvfp4 {

constexpr uint32_t kMxNan = 255u;

// Scale byte of a block whose largest |x| has the fp32 bits m (integer maximum of the magnitudes'
// bits, so that a NaN or an infinity wins).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t m, bool ceil_rule)
{
    const int e = (int)(m >> 23) - 2 + ((ceil_rule && (m & 0x7FFFFFu) > 0x400000u) ? 1 : 0);
    return m >= 0x7F800000u ? kMxNan : (uint32_t)(e > 0 ? e : 0);
}

// 2^(127 - b); 0 for b = 255, so that x * it is 0 or NaN, whose codes the caller drops.
__device__ __forceinline__ float mx_inverse(uint32_t b)
{
    return b == kMxNan ? 0.0f : __uint_as_float((254u - b) << 23);
}

// fp32 value of scale byte b: 2^(b - 127) (b = 0 is subnormal), NaN for 255.
__device__ __forceinline__ float mx_scale_f32(uint32_t b)
{
    return __uint_as_float(b == 0u ? 0x00400000u : b == kMxNan ? 0x7FC00000u : b << 23);
}

// max per unsigned 16-bit half
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

constexpr uint32_t kAbs16x2 = 0x7FFF7FFFu;

// max(|a|, |b|) per bf16 half, NaN if either is, the sign bits left to be masked: one instruction for
// a mask and a maximum.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight bf16 (four words) -> eight E2M1 codes of x * inv.
__device__ __forceinline__ uint32_t mx_codes_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                                    float inv)
{
    const uint32_t u[4] = {a, b, c, d};
    float y[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 p = __fmul2_rn(
            make_float2(__uint_as_float(u[q] << 16), __uint_as_float(u[q] & 0xFFFF0000u)),
            make_float2(inv, inv));
        y[2 * q] = p.x;
        y[2 * q + 1] = p.y;
    }
    return cvt_e2m1x8(y);
}

__device__ __forceinline__ uint32_t mx_codes_f32x8(const uint4 &a, const uint4 &b, float inv)
{
    const float v[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z),
                        __uint_as_float(a.w), __uint_as_float(b.x), __uint_as_float(b.y),
                        __uint_as_float(b.z), __uint_as_float(b.w)};
    float y[8];
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
        const float2 p = __fmul2_rn(make_float2(v[q], v[q + 1]), make_float2(inv, inv));
        y[q] = p.x;
        y[q + 1] = p.y;
    }
    return cvt_e2m1x8(y);
}

// One whole block from memory (16-byte aligned): 32 bf16 / fp32 values -> 16 code bytes and the
// scale byte (floor rule).
__device__ __forceinline__ void mx_encode_bf16(const uint4 *src, uint32_t (&w)[4], uint32_t &sb)
{
    uint4 v[4];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __ldg(src + i);
        m = max_u16x2(m, max_u16x2(max_u16x2(v[i].x & kAbs16x2, v[i].y & kAbs16x2),
                                   max_u16x2(v[i].z & kAbs16x2, v[i].w & kAbs16x2)));
    }
    sb = mx_scale_byte(max(m & 0xFFFFu, m >> 16) << 16, false);
    const float inv = mx_inverse(sb);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = sb == kMxNan ? 0u : mx_codes_bf16x8(v[i].x, v[i].y, v[i].z, v[i].w, inv);
}

__device__ __forceinline__ void mx_encode_f32(const uint4 *src, uint32_t (&w)[4], uint32_t &sb)
{
    uint4 v[8];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = __ldg(src + i);
        m = max(m, max(max(v[i].x & 0x7FFFFFFFu, v[i].y & 0x7FFFFFFFu),
                       max(v[i].z & 0x7FFFFFFFu, v[i].w & 0x7FFFFFFFu)));
    }
    sb = mx_scale_byte(m, false);
    const float inv = mx_inverse(sb);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = sb == kMxNan ? 0u : mx_codes_f32x8(v[2 * i], v[2 * i + 1], inv);
}

} // namespace nvfp4
