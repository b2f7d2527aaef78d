// MXFP4 (E2M1 elements, one E8M0 scale per 32): conversions and argument checks shared by the
// moe_mx4_* translation units.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_ptx.cuh"

// 2^(s - 127); 255 is NaN.
__device__ __forceinline__ float e8m0_value(int s) {
    const uint32_t bits = s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : (uint32_t)s << 23;
    return __uint_as_float(bits);
}

// The scale byte of a block whose largest magnitude has these bits: floor(log2 amax) - 2, biased and
// clamped at 0, straight from the exponent field (a subnormal or zero amax gives 0); an infinity
// or a NaN gives 255.  Magnitudes compare as integers, NaN above all.
__device__ __forceinline__ int e8m0_of_amax(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23);
    return e == 255 ? 255 : max(0, e - 2);
}
// 2^(127 - s), the multiplier that brings a block of scale s into the E2M1 range (s <= 252: a
// power of two with an exact product wherever the result is not far below the smallest code).
__device__ __forceinline__ float e8m0_inverse(int s) { return e8m0_value(254 - s); }

// Eight floats to E2M1 codes, nearest even, saturating at 6: element i at bits 4i.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// Values of eight codes, two to a half2.
__device__ __forceinline__ void e2m1x8_value(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// silu(g) * u with s = exp(-|g| / 2), which neither overflows nor leaves the normal numbers before |g| = 174:
// sigmoid(g) = q^2 / (1 + s^2), q = 1 for g >= 0, s below; multiplied as (g q) (q u) / (1 + s^2), so that nothing
// is lost before the result itself is.  2^x and 1 / x by the approximate instructions (2^-22, 2^-23).
// FULL: the argument's rounding, up to |g| * 2^-24, is put back to first order.  Then h is off by at most
// 17 * 2^-24 of itself (2 (4 + 1) for s^2, 1 + 2 for the denominator's inverse, 4 products), whatever g;
// without, for an h that is rounded to 2^-8, by 2^-19 + |g| 2^-22.  Measured, gate/up of 32768 routes: fp32 in
// full 86.7 us, bf16 without 82.9; both by __expf and __fdividef 84.3 and 82.6, but off by 2 + 1.2 |g| units and 0
// for every g below -87; bf16 by expf and a division 107.
template <bool FULL>
__device__ __forceinline__ float mx4_swiglu(float g, float u) {
    constexpr double LOG2E_HALF = 1.4426950408889634 / 2;
    constexpr float C = (float)LOG2E_HALF, C_LOW = (float)(LOG2E_HALF - (double)C);
    const float a = FULL ? fmaxf(-fabsf(g), -512.f) : -fabsf(g), x = a * C;  // (infinite - infinite below)
    float s, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(x));
    if (FULL) s = fmaf(s * 0.69314718f, fmaf(a, C_LOW, fmaf(a, C, -x)), s);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(s, s, 1.f)));
    const float q = g >= 0.f ? 1.f : s;
    return g * (q * r) * (q * u);
}

// Eight consecutive elements as they are stored (wide loads where `wide`), as floats, and back.
template <int XT>
struct Raw8 {
    uint32_t w[XT == MOE_BF16 ? 4 : 8];
};
template <int XT>
__device__ __forceinline__ Raw8<XT> load_raw8(const void *p, size_t i, bool wide) {
    Raw8<XT> r;
    if (XT == MOE_BF16) {
        const uint16_t *b = (const uint16_t *)p + i;
        if (wide) {
            const uint4 u = *(const uint4 *)b;
            r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) r.w[j] = (uint32_t)b[2 * j] | (uint32_t)b[2 * j + 1] << 16;
        }
    } else {
        const uint32_t *f = (const uint32_t *)p + i;
        if (wide) {
            const uint4 a = *(const uint4 *)f, b = *(const uint4 *)(f + 4);
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
            r.w[XT == MOE_BF16 ? 0 : 4] = b.x; r.w[XT == MOE_BF16 ? 0 : 5] = b.y;
            r.w[XT == MOE_BF16 ? 0 : 6] = b.z; r.w[XT == MOE_BF16 ? 0 : 7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < (XT == MOE_BF16 ? 4 : 8); ++j) r.w[j] = f[j];
        }
    }
    return r;
}
template <int XT>
__device__ __forceinline__ void raw8_floats(const Raw8<XT> &r, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (XT == MOE_BF16) {
            v[2 * j] = __uint_as_float(r.w[j] << 16);
            v[2 * j + 1] = __uint_as_float(r.w[j] & 0xFFFF0000u);
        } else {
            v[2 * j] = __uint_as_float(r.w[XT == MOE_BF16 ? 0 : 2 * j]);
            v[2 * j + 1] = __uint_as_float(r.w[XT == MOE_BF16 ? 0 : 2 * j + 1]);
        }
    }
}
// Bits of the largest magnitude of the eight (as fp32).
template <int XT>
__device__ __forceinline__ uint32_t raw8_amax(const Raw8<XT> &r) {
    if (XT == MOE_BF16) {
        const uint32_t m = 0x7FFF7FFFu;
        const uint32_t a = __vmaxu2(__vmaxu2(r.w[0] & m, r.w[1] & m), __vmaxu2(r.w[2] & m, r.w[3] & m));
        return max(a << 16, a & 0xFFFF0000u);
    }
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < (XT == MOE_BF16 ? 4 : 8); ++j) a = max(a, r.w[j] & 0x7FFFFFFFu);
    return a;
}
template <int XT>
__device__ __forceinline__ void store8(void *p, size_t i, bool wide, const float (&v)[8]) {
    if (XT == MOE_BF16) {
        __nv_bfloat16 *b = (__nv_bfloat16 *)p + i;
        if (wide) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                w[j] = *(const uint32_t *)&h;
            }
            *(uint4 *)b = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = __float2bfloat16(v[j]);
        }
    } else {
        float *f = (float *)p + i;
        if (wide) {
            *(float4 *)f = make_float4(v[0], v[1], v[2], v[3]);
            *(float4 *)(f + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = v[j];
        }
    }
}

// One thread's eight elements of a 32-column block shared by four neighbouring lanes: the block's
// scale byte and the eight codes (element i at bits 4i).  All 32 lanes must call it.
template <int XT>
__device__ __forceinline__ uint32_t mx4_quant8(const Raw8<XT> &r, int &scale) {
    uint32_t amax = raw8_amax<XT>(r);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    scale = e8m0_of_amax(amax);
    if (scale == 255) return 0;
    const float inv = e8m0_inverse(scale);
    float v[8];
    raw8_floats<XT>(r, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv;
    return e2m1x8(v);
}
__device__ __forceinline__ void mx4_dequant8(uint32_t codes, int scale, float (&v)[8]) {
    const float m = e8m0_value(scale);
    uint32_t h[4];
    e2m1x8_value(codes, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*(const __half2 *)&h[j]);
        v[2 * j] = f.x * m;
        v[2 * j + 1] = f.y * m;
    }
}
