// MXFP4 (E2M1 elements, one E8M0 scale per 32): conversions and argument checks shared by the
// moe_mx4_* translation units.
#pragma once

#include <cuda_bf16.h>

#include "moe_ptx.cuh"

// 2^(s - 127); 255 is NaN.
__device__ __forceinline__ float e8m0_value(int s) {
    const uint32_t bits = s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : (uint32_t)s << 23;
    return __uint_as_float(bits);
}

// The scale byte of a block whose largest magnitude is amax: floor(log2 amax) - 2, biased and
// clamped at 0, straight from the exponent field (a subnormal or zero amax gives 0); an infinity
// or a NaN gives 255.
__device__ __forceinline__ int e8m0_of_amax(float amax) {
    const int e = (int)(__float_as_uint(amax) >> 23);
    return e == 255 ? 255 : max(0, e - 2);
}
// 2^(127 - s), the multiplier that brings a block of scale s into the E2M1 range (s <= 252: a
// power of two with an exact product wherever the result is not far below the smallest code).
__device__ __forceinline__ float e8m0_inverse(int s) { return e8m0_value(254 - s); }

// Two floats to E2M1 codes, nearest even, saturating at 6: lo in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Value of a 4-bit code: doubled magnitudes 0 1 2 3 4 6 8 12 as nibbles of a constant.
__device__ __forceinline__ float e2m1_value(uint32_t code) {
    const float m = 0.5f * (float)((0xC8643210u >> (4 * (code & 7))) & 15);
    return code & 8 ? -m : m;
}

// Eight consecutive elements as floats (wide loads where `wide`).
template <int XT>
__device__ __forceinline__ void load8(const void *p, size_t i, bool wide, float (&v)[8]) {
    if (XT == MOE_BF16) {
        const __nv_bfloat16 *b = (const __nv_bfloat16 *)p + i;
        if (wide) {
            const uint4 u = *(const uint4 *)b;
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __bfloat162float(b[j]);
        }
    } else {
        const float *f = (const float *)p + i;
        if (wide) {
            const float4 a = *(const float4 *)f, b = *(const float4 *)(f + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = f[j];
        }
    }
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
__device__ __forceinline__ uint32_t mx4_quant8(const float (&v)[8], int &scale) {
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        amax = fmaxf(amax, fabsf(v[j]));
        bad |= !(fabsf(v[j]) <= 3.402823466e38f);  // fmaxf drops a NaN
    }
    if (bad) amax = __uint_as_float(0x7F800000u);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    scale = e8m0_of_amax(amax);
    if (scale == 255) return 0;
    const float inv = e8m0_inverse(scale);
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) c |= e2m1x2(v[2 * j] * inv, v[2 * j + 1] * inv) << (8 * j);
    return c;
}
__device__ __forceinline__ void mx4_dequant8(uint32_t codes, int scale, float (&v)[8]) {
    const float m = e8m0_value(scale);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e2m1_value((codes >> (4 * j)) & 15) * m;
}
