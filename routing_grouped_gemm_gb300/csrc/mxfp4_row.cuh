// Microscaled 4-bit floating point (MXFP4 of the Open Compute Project's
// Microscaling Formats specification 1.0): 32 consecutive values of a row
// share one power-of-two scale (e8m0: byte b stands for 2^(b - 127)) and each
// value is an e2m1 code (sign and 0, 0.5, 1, 1.5, 2, 3, 4, 6).
//
// For a block with largest magnitude m, the scale is 2^e with
//   e = floor(log2 m) - 2  (2: exponent of the largest e2m1 binade),
// at least -127, and the codes are x 2^-e to the nearest e2m1 value, ties to
// the even code, saturating at 6.  floor(log2 m) is m's binary32 exponent
// field, so the scale byte is that field less 2 (0 where that is negative:
// zero, subnormal or tiny m), and x 2^-e is one exact multiplication by a
// power of two: scale and codes are the same bits however they are computed.
// A block that holds a NaN or an infinity gets scale byte 255 (e8m0's NaN)
// and codes 0, so all of its 32 values read back as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <stdint.h>

namespace moe {

constexpr uint32_t kMxNan = 255u;

// Scale byte of a block; amax_bits: the largest |x| of the block as its bits
// (a NaN's are above infinity's, so an integer maximum finds either).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? kMxNan : e > 2u ? e - 2u : 0u;
}

// 2^-e for scale byte b = e + 127 <= 252; 0 for a NaN block, whose codes are 0.
__device__ __forceinline__ float mx_inv_scale(uint32_t b) {
    return __uint_as_float(b == kMxNan ? 0u : (254u - b) << 23);
}

// 2^e for scale byte b; byte 0 is the subnormal 2^-127, byte 255 a NaN.
__device__ __forceinline__ float mx_scale(uint32_t b) {
    return __uint_as_float(b == kMxNan ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Codes of 8 consecutive values, the first in the lowest 4 bits.  A NaN block
// (inv = 0) gets codes 0 whatever its values are.
__device__ __forceinline__ uint32_t mx_codes8(const float (&f)[8], float inv) {
    if (inv == 0.f) return 0u;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(f[2 * i] * inv, f[2 * i + 1] * inv),
                                                __NV_E2M1, cudaRoundNearest)
             << (8 * i);
    return c;
}

// The value of e2m1 code c (0..15) as binary32: codes of magnitude 2..7 have
// exponent field c / 2 and one mantissa bit, code 1 is 0.5.
__device__ __forceinline__ float mx_value(uint32_t c) {
    const uint32_t m = c & 7u;
    const uint32_t mag = m >= 2u ? ((m >> 1) + 126u) << 23 | (m & 1u) << 22 : m ? 0x3f000000u : 0u;
    return __uint_as_float(mag | (c & 8u) << 28);
}

// 8 consecutive values of a bf16 or fp32 row.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&f)[8]) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
    const __nv_bfloat162 *h2 = reinterpret_cast<const __nv_bfloat162 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __low2float(h2[i]);
        f[2 * i + 1] = __high2float(h2[i]);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Largest |x| (as bits) of a block whose 4 x 8 values four neighbouring lanes
// hold; every lane of the warp takes part.
__device__ __forceinline__ uint32_t mx_amax_quad(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// One bf16 row by one warp (the quantising dispatch): lane j < n_dst holds in
// my_row the destination row of copy j (-1: none); codes go to rows my_row of
// dst ([*, cols / 2] bytes), scales to rows my_row of sf ([*, cols / 32]).
// Four lanes hold a block; the warp reads 256 values a step.
__device__ __forceinline__ void quantize_row_mxfp4_warp(const __nv_bfloat16 *__restrict__ x,
                                                        int cols, int my_row, int n_dst,
                                                        uint8_t *__restrict__ dst,
                                                        uint8_t *__restrict__ sf, int lane) {
    for (int c0 = 0; c0 < cols; c0 += 256) {
        const int c = c0 + lane * 8;
        float f[8] = {};
        if (c < cols) load8(x + c, f);
        const uint32_t b = mx_scale_byte(mx_amax_quad(f));
        const uint32_t q = mx_codes8(f, mx_inv_scale(b));
        for (int j = 0; j < n_dst; ++j) {
            const int r = __shfl_sync(0xffffffffu, my_row, j);
            if (r < 0 || c >= cols) continue;
            *reinterpret_cast<uint32_t *>(dst + (size_t)r * (cols / 2) + c / 2) = q;
            if ((lane & 3) == 0) sf[(size_t)r * (cols / 32) + c / 32] = (uint8_t)b;
        }
    }
}

}  // namespace moe
