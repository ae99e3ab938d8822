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
constexpr int MX_UNROLL = 4;

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

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}

// Every value is exact in bf16 as in fp32 (two significant bits, exponents of
// the binary32 range) but beyond scale byte 252, which the quantiser never
// writes: there 6 * 2^126 and more round to infinity as binary32 does.
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
        q[u] = i < n8 ? codes[i] : 0u;
        b[u] = i < n8 ? scale[i >> 2] : 0u;
    }
#pragma unroll
    for (int u = 0; u < MX_UNROLL; ++u) {
        const long long i = base + u * 256;
        if (i >= n8) continue;
        const float s = mx_scale(b[u]);
        float f[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) f[v] = mx_value((q[u] >> (4 * v)) & 15u) * s;
        store8(dst + i * 8, f);
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
    quantize_row_mxfp4_warp(src + (size_t)t * cols, cols, my_row, k, dst, scale, lane);
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
