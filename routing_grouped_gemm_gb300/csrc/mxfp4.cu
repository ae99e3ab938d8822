// Rows to MXFP4 and back (the arithmetic is in mxfp4_row.cuh).
//
// Both directions move each value once and compute almost nothing, so they
// are bound by memory: 4.25 bits per value on the 4-bit side and 16 or 32 on
// the other.  cols is a multiple of 32, so blocks never straddle rows and the
// whole tensor is one run of blocks; four neighbouring lanes hold a block,
// which makes every load a contiguous 512 or 1024 bytes of a warp and the
// block's maximum two shuffles away.
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "mxfp4_row.cuh"

namespace moe {
namespace {

// 8-value pieces of a thread that are in flight together.
#ifndef MOE_MXQ_UNROLL
#define MOE_MXQ_UNROLL 4
#endif
constexpr int MX_UNROLL = MOE_MXQ_UNROLL;

template <typename T>
__global__ void __launch_bounds__(256)
quantize_rows_mxfp4_kernel(const T *__restrict__ src, long long n8, uint32_t *__restrict__ dst,
                           uint8_t *__restrict__ scale) {
    griddep_launch_dependents();  // the next kernel may be scheduled now
    griddep_wait();               // every input of this kernel is complete
    const long long base = (long long)blockIdx.x * (256 * MX_UNROLL) + threadIdx.x;
    float f[MX_UNROLL][8];
#pragma unroll
    for (int u = 0; u < MX_UNROLL; ++u) {
        const long long i = base + u * 256;
#pragma unroll
        for (int v = 0; v < 8; ++v) f[u][v] = 0.f;
        if (i < n8) load8(src + i * 8, f[u]);
    }
#pragma unroll
    for (int u = 0; u < MX_UNROLL; ++u) {
        const long long i = base + u * 256;
        const uint32_t b = mx_scale_byte(mx_amax_quad(f[u]));
        if (i >= n8) continue;  // whole quads: n8 is a multiple of 4
        dst[i] = mx_codes8(f[u], mx_inv_scale(b));
        if ((i & 3) == 0) scale[i >> 2] = (uint8_t)b;
    }
}

// 8 values held as bf16 (two to a word) to a bf16 or an fp32 row.
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const uint32_t (&w)[4]) {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(float *p, const uint32_t (&w)[4]) {
    uint4 *o = reinterpret_cast<uint4 *>(p);
    __stcs(o, make_uint4(w[0] << 16, w[0] & 0xffff0000u, w[1] << 16, w[1] & 0xffff0000u));
    __stcs(o + 1, make_uint4(w[2] << 16, w[2] & 0xffff0000u, w[3] << 16, w[3] & 0xffff0000u));
}

// Every value is exact in bf16 as in fp32 (two significant bits, exponents of
// the binary32 range) but beyond scale byte 252, which the quantiser never
// writes: there a value above the range becomes infinite.
template <typename T>
__global__ void __launch_bounds__(256)
dequantize_rows_mxfp4_kernel(const uint32_t *__restrict__ codes, const uint8_t *__restrict__ scale,
                             long long n8, T *__restrict__ dst) {
    griddep_launch_dependents();
    griddep_wait();
    const long long base = (long long)blockIdx.x * (256 * MX_UNROLL) + threadIdx.x;
    uint32_t q[MX_UNROLL], b[MX_UNROLL];
#pragma unroll
    for (int u = 0; u < MX_UNROLL; ++u) {
        const long long i = base + u * 256;
        q[u] = i < n8 ? __ldcs(codes + i) : 0u;
        b[u] = i < n8 ? scale[i >> 2] : 0u;
    }
#pragma unroll
    for (int u = 0; u < MX_UNROLL; ++u) {
        const long long i = base + u * 256;
        if (i >= n8) continue;
        uint32_t w[4];
        mx_values8(q[u], mx_scale_bf16x2(b[u]), w);
        store8(dst + i * 8, w);
    }
}

// One warp per token: its codes and scales to the k dispatched rows.
__global__ void __launch_bounds__(256)
dispatch_rows_mxfp4_kernel(const __nv_bfloat16 *__restrict__ src, long long rows, int cols,
                           const int *__restrict__ row_of, int k, uint8_t *__restrict__ dst,
                           uint8_t *__restrict__ scale) {
    griddep_launch_dependents();
    griddep_wait();
    const long long t = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (t >= rows) return;
    const int my_row = lane < k ? row_of[(size_t)t * k + lane] : -1;
    quantize_row_mxfp4_warp(src + (size_t)t * cols, cols, 0, 256, my_row, k, dst, scale, lane);
}

bool grid_of(long long n8, unsigned *blocks) {
    const long long b = (n8 + 256 * MX_UNROLL - 1) / (256 * MX_UNROLL);
    *blocks = (unsigned)b;
    return b <= 0x7fffffffLL;
}

}  // namespace

cudaError_t launch_quantize_rows_mxfp4(const void *src, int64_t rows, int cols, int is_bf16,
                                       uint8_t *dst, uint8_t *scale, cudaStream_t stream) {
    if (rows == 0) return cudaSuccess;
    const long long n8 = (long long)rows * (cols / 8);
    unsigned blocks;
    if (cols % 32 || !grid_of(n8, &blocks)) return cudaErrorInvalidValue;
    const cudaError_t e =
        is_bf16 ? launch_pdl(quantize_rows_mxfp4_kernel<__nv_bfloat16>, dim3(blocks), dim3(256), 0,
                             stream, (const __nv_bfloat16 *)src, n8, (uint32_t *)dst, scale)
                : launch_pdl(quantize_rows_mxfp4_kernel<float>, dim3(blocks), dim3(256), 0, stream,
                             (const float *)src, n8, (uint32_t *)dst, scale);
    if (e == cudaSuccess) count_launch();
    return e;
}

cudaError_t launch_dequantize_rows_mxfp4(const uint8_t *codes, const uint8_t *scale, int64_t rows,
                                         int cols, int is_bf16, void *dst, cudaStream_t stream) {
    if (rows == 0) return cudaSuccess;
    const long long n8 = (long long)rows * (cols / 8);
    unsigned blocks;
    if (cols % 32 || !grid_of(n8, &blocks)) return cudaErrorInvalidValue;
    const cudaError_t e =
        is_bf16 ? launch_pdl(dequantize_rows_mxfp4_kernel<__nv_bfloat16>, dim3(blocks), dim3(256),
                             0, stream, (const uint32_t *)codes, scale, n8, (__nv_bfloat16 *)dst)
                : launch_pdl(dequantize_rows_mxfp4_kernel<float>, dim3(blocks), dim3(256), 0, stream,
                             (const uint32_t *)codes, scale, n8, (float *)dst);
    if (e == cudaSuccess) count_launch();
    return e;
}

cudaError_t launch_dispatch_rows_mxfp4(const void *src, int64_t rows, int cols, const int *row_of,
                                       int k, uint8_t *dst, uint8_t *scale, cudaStream_t stream) {
    if (rows == 0) return cudaSuccess;
    if (cols % 32 || k > 32) return cudaErrorInvalidValue;
    const unsigned blocks = (unsigned)((rows + 7) / 8);
    const cudaError_t e = launch_pdl(dispatch_rows_mxfp4_kernel, dim3(blocks), dim3(256), 0, stream,
                                     (const __nv_bfloat16 *)src, (long long)rows, cols, row_of, k,
                                     dst, scale);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace moe
