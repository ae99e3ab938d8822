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

// 2^e for scale byte b as two bf16 (byte 0 is the subnormal 2^-127, 255 a NaN).
__device__ __forceinline__ __nv_bfloat162 mx_scale_bf16x2(uint32_t b) {
    const uint32_t h = b == kMxNan ? 0x7fc0u : b == 0u ? 0x0040u : b << 7;
    const uint32_t w = h | h << 16;
    return *reinterpret_cast<const __nv_bfloat162 *>(&w);
}

// The values of 8 codes (the first in the lowest 4 bits) times 2^e, as bf16, two
// to a word: exact but where 2^e 6 leaves the range.  The 8 magnitudes of e2m1
// are a table of 8 bytes for bf16's upper byte and one for its lower: a byte
// permute looks four codes up at once (about 3 instructions a value with the
// product, against 10 when each is put together by itself).
__device__ __forceinline__ void mx_values8(uint32_t q, __nv_bfloat162 scale, uint32_t (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t c = q >> (16 * i), m = c & 0x7777u;
        //             6 4 3 2          1.5 1 0.5 0
        const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, m);
        const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, m);
        o[2 * i] = __byte_perm(lo, hi, 0x5140u) | (c & 0x8u) << 12 | (c & 0x80u) << 24;
        o[2 * i + 1] = __byte_perm(lo, hi, 0x7362u) | (c & 0x800u) << 4 | (c & 0x8000u) << 16;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&o[i]), scale);
        o[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
}

// 8 consecutive values of a bf16 or fp32 row.
__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
    const __nv_bfloat162 *h2 = reinterpret_cast<const __nv_bfloat162 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __low2float(h2[i]);
        f[2 * i + 1] = __high2float(h2[i]);
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&f)[8]) {
    unpack8(__ldcs(reinterpret_cast<const uint4 *>(p)), f);
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

// One bf16 row by one warp (the quantising dispatch), or its 256 values from
// c_first on and every c_step on from there by each of several warps: lane j <
// n_dst holds in my_row the destination row of copy j (-1: none); codes go to
// rows my_row of dst ([*, cols / 2] bytes), scales to rows my_row of sf
// ([*, cols / 32]).  Four lanes hold a block; the warp takes 256 values at a
// time and has the loads of kMxBatch of those in flight before it uses the
// first: with one, each step of a row waited for memory in turn.
constexpr int kMxBatch = 8;
static_assert(kMxBatch == 8, "two stores of four steps' scales");

__device__ __forceinline__ void quantize_row_mxfp4_warp(const __nv_bfloat16 *__restrict__ x,
                                                        int cols, int c_first, int c_step,
                                                        int my_row, int n_dst,
                                                        uint8_t *__restrict__ dst,
                                                        uint8_t *__restrict__ sf, int lane) {
    const uint4 *xv = reinterpret_cast<const uint4 *>(x);
    for (int c0 = c_first; c0 < cols; c0 += c_step * kMxBatch) {
        uint4 raw[kMxBatch];
#pragma unroll
        for (int u = 0; u < kMxBatch; ++u) {
            const int c = c0 + u * c_step + lane * 8;
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            if (c < cols) raw[u] = __ldcs(xv + c / 8);
        }
        uint32_t q[kMxBatch], b[kMxBatch];
#pragma unroll
        for (int u = 0; u < kMxBatch; ++u) {
            float f[8];
            unpack8(raw[u], f);
            b[u] = mx_scale_byte(mx_amax_quad(f));
            q[u] = mx_codes8(f, mx_inv_scale(b[u]));
        }
        // a block's lanes all hold its scale: each stores that of another step
        const int i = lane & 3, cs = c0 + i * c_step + (lane & ~3) * 8;
        const uint32_t b0 = i & 2 ? (i & 1 ? b[3] : b[2]) : (i & 1 ? b[1] : b[0]);
        const uint32_t b1 = i & 2 ? (i & 1 ? b[7] : b[6]) : (i & 1 ? b[5] : b[4]);
        for (int j = 0; j < n_dst; ++j) {
            const int r = __shfl_sync(0xffffffffu, my_row, j);
            if (r < 0) continue;
            uint8_t *qr = dst + (size_t)r * (cols / 2), *sr = sf + (size_t)r * (cols / 32);
#pragma unroll
            for (int u = 0; u < kMxBatch; ++u) {
                const int c = c0 + u * c_step + lane * 8;
                if (c >= cols) continue;
                *reinterpret_cast<uint32_t *>(qr + c / 2) = q[u];
            }
            if (cs < cols) sr[cs / 32] = (uint8_t)b0;
            if (cs + 4 * c_step < cols) sr[(cs + 4 * c_step) / 32] = (uint8_t)b1;
        }
    }
}

}  // namespace moe
