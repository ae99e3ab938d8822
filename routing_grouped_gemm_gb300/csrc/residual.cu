// The norms around a block, fused with its gate, dropout and residual sum.
//
// Per token (row of D values), with resid r, branch output y:
//   v = y                                    without a post gain,
//   v = y rsqrt(mean(y^2) + eps) post        with one;
//   s = res_scale r + branch_scale gate keep v          (the new residual)
//   n = s rsqrt(mean(s^2) + eps) pre                    (the next block's input)
// keep is 0 or 1 / (1 - p) from a counter-based generator (keep_word below),
// so no mask is stored: forward and gradient derive it from (seed, offset).
// All arithmetic is fp32; s and n are rounded once each, and n is the norm of
// the unrounded s.
//
// Every element is touched a fixed few times, so the passes are bound by HBM:
// forward 4 T D elements (r, y in; s, n out), gradient 6 (s, y, ds, dn in; dr,
// dy out).  One CTA owns a row at a time and keeps it in registers between the
// row sums, so nothing is read twice.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

enum { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_TOKEN = 2, GATE_ELEMENT = 3 };

// ---------------------------------------------------------------------
// rows in vectors of 8 elements
// ---------------------------------------------------------------------
template <bool BF16> struct Pack;
template <> struct Pack<true> {
    uint4 a;
};
template <> struct Pack<false> {
    uint4 a, b;
};

template <bool BF16>
__device__ __forceinline__ Pack<BF16> load8(const void *p, size_t vec) {
    Pack<BF16> r;
    if constexpr (BF16) {
        r.a = static_cast<const uint4 *>(p)[vec];
    } else {
        r.a = static_cast<const uint4 *>(p)[2 * vec];
        r.b = static_cast<const uint4 *>(p)[2 * vec + 1];
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const Pack<BF16> &p, float (&f)[8]) {
    if constexpr (BF16) {
        const uint32_t w[4] = {p.a.x, p.a.y, p.a.z, p.a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const uint32_t w[8] = {p.a.x, p.a.y, p.a.z, p.a.w, p.b.x, p.b.y, p.b.z, p.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void *p, size_t vec, const float (&f)[8]) {
    if constexpr (BF16) {
        uint4 o;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        static_cast<uint4 *>(p)[vec] = o;
    } else {
        static_cast<float4 *>(p)[2 * vec] = make_float4(f[0], f[1], f[2], f[3]);
        static_cast<float4 *>(p)[2 * vec + 1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// ---------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------
// Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011).  Counter (i, offset), key seed; i
// numbers the T D / 8 vectors of 8 elements.
__device__ __forceinline__ uint4 philox(uint64_t i, uint64_t offset, uint64_t seed) {
    uint32_t c0 = (uint32_t)i, c1 = (uint32_t)(i >> 32);
    uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xd2511f53u * c0, p1 = (uint64_t)0xcd9e8d57u * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)p1;
        c3 = (uint32_t)p0;
        k0 += 0x9e3779b9u;
        k1 += 0xbb67ae85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// What a launch knows of the dropout: an element stays when its 16-bit half
// word is at least cut (0: no dropout), and is then multiplied by `scale`.
struct Drop {
    const int64_t *rng;  // seed, offset (device)
    uint32_t cut;
    float scale;
};

// f[e] *= keep factor: half words of the vector's four words, low half first.
__device__ __forceinline__ void drop8(float (&f)[8], uint64_t vec, const Drop &d, uint64_t seed,
                                      uint64_t offset) {
    const uint4 w = philox(vec, offset, seed);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = (u[i] & 0xffffu) >= d.cut ? f[2 * i] * d.scale : 0.f;
        f[2 * i + 1] = (u[i] >> 16) >= d.cut ? f[2 * i + 1] * d.scale : 0.f;
    }
}

// ---------------------------------------------------------------------
// row sums over a CTA
// ---------------------------------------------------------------------
// Sums v[0..N) over the CTA's threads; every thread gets them.  One barrier:
// `slot` must be another buffer ([N][32] floats) than the call before's.  The
// order is fixed by the block size.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if (nwarps == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) slot[n * 32 + warp] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        v[n] = lane < nwarps ? slot[n * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    }
}

// ---------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------
struct ForwardArgs {
    const void *resid, *y, *post, *gate, *pre;
    void *y_out, *resid_out, *norm_out;
    Drop drop;
    float eps, res_scale, branch_scale;
    int T, D, gate_kind;
    // the combine in front (COMBINE): y[t] = sum_j topk_w[t, j] y_perm[row_of[t, j]]
    const int *row_of;
    const float *topk_w;
    int k;
    long long rows_alloc;
    int *status;
};

template <bool BF16>
__device__ __forceinline__ void expert_row8(const void *y_perm, size_t vec, float (&f)[8]) {
    if constexpr (BF16) {  // fp16 rows
        const uint4 q = __ldcs(static_cast<const uint4 *>(y_perm) + vec);
        const __half2 *h = reinterpret_cast<const __half2 *>(&q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(h[i]);
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    } else {
        unpack8<false>(load8<false>(y_perm, vec), f);
    }
}

// NV vectors of 8 per thread: vector tid + i blockDim of the row.
template <bool BF16, int NV, bool COMBINE>
__global__ void __launch_bounds__(1024)
residual_norm_kernel(const ForwardArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float s_sum[2][32];
    __shared__ int s_row[32];
    __shared__ float s_w[32];
    const int V = a.D / 8, tid = threadIdx.x;
    const float inv_d = 1.f / (float)a.D;
    const bool branch = COMBINE || a.y;
    uint64_t seed = 0, offset = 0;
    if (a.drop.cut) {
        seed = (uint64_t)a.drop.rng[0];
        offset = (uint64_t)a.drop.rng[1];
    }
    int turn = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t base = (size_t)t * V;
        if constexpr (COMBINE) {
            __syncthreads();  // the row before is done with s_row
            if (tid < a.k) {
                int r = a.row_of[(size_t)t * a.k + tid];
                if (r < -1 || (long long)r >= a.rows_alloc) {
                    raise_flag(a.status, FLAG_BAD_ROUTING);
                    r = -1;
                }
                s_row[tid] = r;
                s_w[tid] = a.topk_w[(size_t)t * a.k + tid];
            }
            __syncthreads();
        }
        float s[NV][8], y[NV][8];
        float sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * blockDim.x;
#pragma unroll
            for (int e = 0; e < 8; ++e) s[i][e] = y[i][e] = 0.f;
            if (v >= V) continue;
            unpack8<BF16>(load8<BF16>(a.resid, base + v), s[i]);
            if constexpr (COMBINE) {
                for (int j = 0; j < a.k; ++j) {
                    if (s_row[j] < 0) continue;
                    float f[8];
                    expert_row8<BF16>(a.y, (size_t)s_row[j] * V + v, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[i][e] = fmaf(s_w[j], f[e], y[i][e]);
                }
                if (a.y_out) store8<BF16>(a.y_out, base + v, y[i]);
            } else if (branch) {
                unpack8<BF16>(load8<BF16>(a.y, base + v), y[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[0] = fmaf(y[i][e], y[i][e], sum[0]);
        }
        if (branch) {
            float r1 = 1.f;
            if (a.post) {
                block_sum<1>(sum, s_sum[turn]);
                turn ^= 1;
                r1 = rsqrtf(fmaf(sum[0], inv_d, a.eps));
            }
            const float gt = a.gate_kind == GATE_TOKEN ? static_cast<const float *>(a.gate)[t] : 1.f;
            sum[0] = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = tid + i * blockDim.x;
                if (v >= V) continue;
                float g[8];
                if (a.post) {
                    unpack8<BF16>(load8<BF16>(a.post, v), g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[i][e] = y[i][e] * r1 * g[e];
                }
                if (a.drop.cut) drop8(y[i], base + v, a.drop, seed, offset);
                if (a.gate_kind == GATE_CHANNEL || a.gate_kind == GATE_ELEMENT) {
                    unpack8<BF16>(load8<BF16>(a.gate, a.gate_kind == GATE_CHANNEL ? v : base + v), g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[i][e] *= g[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[i][e] = fmaf(a.res_scale, s[i][e], a.branch_scale * (gt * y[i][e]));
                store8<BF16>(a.resid_out, base + v, s[i]);
            }
        }
        if (!a.pre) continue;
        sum[0] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[0] = fmaf(s[i][e], s[i][e], sum[0]);
        block_sum<1>(sum, s_sum[turn]);
        turn ^= 1;
        const float r2 = rsqrtf(fmaf(sum[0], inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * blockDim.x;
            if (v >= V) continue;
            float g[8];
            unpack8<BF16>(load8<BF16>(a.pre, v), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] *= s[i][e] * r2;
            store8<BF16>(a.norm_out, base + v, g);
        }
    }
}

// ---------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------
struct BackwardArgs {
    const void *s, *y, *post, *gate, *pre, *ds_out, *dn;
    void *dresid, *dy, *dgate;
    float *part;  // [3][gridDim.x][D]: this CTA's sums for dpre, dpost, dgate (channel)
    Drop drop;
    float eps, res_scale, branch_scale;
    int T, D, gate_kind;
};

// With r1, r2 the rows' rsqrt factors and gp = dn pre:
//   ds = ds_out + r2 gp - c s,  c = r2^3 mean(gp s)
//   u = branch_scale keep ds;  dgate = u v;  dv = gate u
//   dy = r1 (dv post - y r1^2 mean(dv post y))
// ds is linear in two row sums that are not known yet, so with
// q = branch_scale keep post y,
//   sum(ds q) = sum(ds_out q) + r2 sum(gp q) - c sum(s q)
// and every sum of the row comes out of ONE reduction.  (mean(dv post y) is
// that sum with the gate inside q, or times the token's gate.)
template <bool BF16, int NV>
__global__ void __launch_bounds__(1024)
residual_norm_backward_kernel(const BackwardArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float s_sum[2][6 * 32];
    const int V = a.D / 8, tid = threadIdx.x;
    const float inv_d = 1.f / (float)a.D;
    const bool branch = a.y;
    const bool elem_gate = a.gate_kind == GATE_CHANNEL || a.gate_kind == GATE_ELEMENT;
    uint64_t seed = 0, offset = 0;
    if (a.drop.cut) {
        seed = (uint64_t)a.drop.rng[0];
        offset = (uint64_t)a.drop.rng[1];
    }
    float dpre[NV][8], dpost[NV][8], dgate[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dpre[i][e] = dpost[i][e] = dgate[i][e] = 0.f;

    int turn = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const size_t base = (size_t)t * V;
        const float gt = a.gate_kind == GATE_TOKEN ? static_cast<const float *>(a.gate)[t] : 1.f;
        // what is read of element e of vector v, and what follows from it
        auto read = [&](int v, float (&s)[8], float (&dso)[8], float (&dn)[8], float (&gp)[8],
                        float (&y)[8], float (&post)[8], float (&gate)[8], float (&keep)[8]) {
            unpack8<BF16>(load8<BF16>(a.s, base + v), s);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dso[e] = dn[e] = gp[e] = y[e] = 0.f;
                post[e] = gate[e] = 1.f;
                keep[e] = a.branch_scale;
            }
            if (a.ds_out) unpack8<BF16>(load8<BF16>(a.ds_out, base + v), dso);
            if (a.pre) {
                unpack8<BF16>(load8<BF16>(a.dn, base + v), dn);
                unpack8<BF16>(load8<BF16>(a.pre, v), gp);
#pragma unroll
                for (int e = 0; e < 8; ++e) gp[e] *= dn[e];
            }
            if (branch) {
                unpack8<BF16>(load8<BF16>(a.y, base + v), y);
                if (a.post) unpack8<BF16>(load8<BF16>(a.post, v), post);
                if (elem_gate)
                    unpack8<BF16>(load8<BF16>(a.gate, a.gate_kind == GATE_CHANNEL ? v : base + v),
                                  gate);
                if (a.drop.cut) drop8(keep, base + v, a.drop, seed, offset);
            }
        };
        float m[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * blockDim.x;
            if (v >= V) continue;
            float s[8], dso[8], dn[8], gp[8], y[8], post[8], gate[8], keep[8];
            read(v, s, dso, dn, gp, y, post, gate, keep);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float q = keep[e] * gate[e] * post[e] * y[e];
                m[0] = fmaf(s[e], s[e], m[0]);
                m[1] = fmaf(gp[e], s[e], m[1]);
                m[2] = fmaf(y[e], y[e], m[2]);
                m[3] = fmaf(dso[e], q, m[3]);
                m[4] = fmaf(gp[e], q, m[4]);
                m[5] = fmaf(s[e], q, m[5]);
            }
        }
        block_sum<6>(m, s_sum[turn]);
        const float r2 = a.pre ? rsqrtf(fmaf(m[0], inv_d, a.eps)) : 0.f;
        const float c = r2 * r2 * r2 * (m[1] * inv_d);
        const float r1 = a.post ? rsqrtf(fmaf(m[2], inv_d, a.eps)) : 1.f;
        const float dot = m[3] + r2 * m[4] - c * m[5];  // sum(ds q)
        const float c1 = a.post ? r1 * r1 * (gt * dot * inv_d) : 0.f;
        if (a.gate_kind == GATE_TOKEN && tid == 0) static_cast<float *>(a.dgate)[t] = r1 * dot;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * blockDim.x;
            if (v >= V) continue;
            float s[8], dso[8], dn[8], gp[8], y[8], post[8], gate[8], keep[8], o[8];
            read(v, s, dso, dn, gp, y, post, gate, keep);
            float dg[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float ds = dso[e] + (r2 * gp[e] - c * s[e]);
                dpre[i][e] = fmaf(dn[e], s[e] * r2, dpre[i][e]);
                const float u = keep[e] * ds, yr = y[e] * r1;
                dg[e] = u * (yr * post[e]);
                dgate[i][e] += dg[e];
                const float dv = u * gate[e] * gt;
                dpost[i][e] = fmaf(dv, yr, dpost[i][e]);
                s[e] = branch ? a.res_scale * ds : ds;
                o[e] = r1 * (dv * post[e] - y[e] * c1);
            }
            store8<BF16>(a.dresid, base + v, s);
            if (branch) store8<BF16>(a.dy, base + v, o);
            if (a.gate_kind == GATE_ELEMENT) store8<BF16>(a.dgate, base + v, dg);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = tid + i * blockDim.x;
        if (v >= V) continue;
        float *p = a.part + (size_t)blockIdx.x * a.D;
        const size_t plane = (size_t)gridDim.x * a.D;
        if (a.pre) store8<false>(p, v, dpre[i]);
        if (a.post) store8<false>(p + plane, v, dpost[i]);
        if (a.gate_kind == GATE_CHANNEL) store8<false>(p + 2 * plane, v, dgate[i]);
    }
}

// out[c] = sum over the CTAs' parts, in a fixed order.  blockIdx.y: which sum.
struct FinishArgs {
    const float *part;
    float *out[3];
    int parts, D;
};

constexpr int FIN_COLS = 32, FIN_ROWS = 16;
__global__ void __launch_bounds__(FIN_COLS *FIN_ROWS)
residual_finish_kernel(const FinishArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float s[FIN_ROWS][FIN_COLS];
    float *out = blockIdx.y == 0 ? a.out[0] : blockIdx.y == 1 ? a.out[1] : a.out[2];
    if (!out) return;
    const int c = blockIdx.x * FIN_COLS + threadIdx.x, r = threadIdx.y;
    const float *p = a.part + (size_t)blockIdx.y * a.parts * a.D;
    float sum = 0.f;
    if (c < a.D)
        for (int i = r; i < a.parts; i += FIN_ROWS) sum += p[(size_t)i * a.D + c];
    s[r][threadIdx.x] = sum;
    __syncthreads();
    if (r == 0 && c < a.D) {
#pragma unroll
        for (int i = 1; i < FIN_ROWS; ++i) sum += s[i][threadIdx.x];
        out[c] = sum;
    }
}

// Threads and vectors per thread for rows of V vectors.
void row_shape(int V, int *threads, int *nv) {
    *nv = V <= 1024 ? 1 : V <= 2048 ? 2 : 4;
    const int n = (V + *nv - 1) / *nv;
    *threads = (n + 31) / 32 * 32;
}

Drop make_drop(const ResidualNorm &r) {
    Drop d;
    d.rng = r.rng;
    d.cut = (uint32_t)r.drop_cut;
    d.scale = 65536.f / (float)(65536 - r.drop_cut);
    return d;
}

template <bool COMBINE>
cudaError_t forward(const ResidualNorm &r, const ForwardArgs &a, cudaStream_t stream) {
    int threads, nv;
    row_shape(r.D / 8, &threads, &nv);
    auto kernel = r.is_bf16 ? (nv == 1   ? residual_norm_kernel<true, 1, COMBINE>
                               : nv == 2 ? residual_norm_kernel<true, 2, COMBINE>
                                         : residual_norm_kernel<true, 4, COMBINE>)
                            : (nv == 1   ? residual_norm_kernel<false, 1, COMBINE>
                               : nv == 2 ? residual_norm_kernel<false, 2, COMBINE>
                                         : residual_norm_kernel<false, 4, COMBINE>);
    const int grid = std::min(r.T, std::max(1, sm_count()) * std::max(1, 2048 / threads));
    const cudaError_t err = launch_pdl(kernel, dim3(grid), dim3(threads), 0, stream, a);
    if (err == cudaSuccess) count_launch();
    return err;
}

ForwardArgs forward_args(const ResidualNorm &r, const void *resid, void *resid_out, void *norm_out) {
    ForwardArgs a = {};
    a.resid = resid;
    a.post = r.post;
    a.gate = r.gate;
    a.pre = r.pre;
    a.resid_out = resid_out;
    a.norm_out = norm_out;
    a.drop = make_drop(r);
    a.eps = r.eps;
    a.res_scale = r.res_scale;
    a.branch_scale = r.branch_scale;
    a.T = r.T;
    a.D = r.D;
    a.gate_kind = r.gate_kind;
    return a;
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNorm &r, const void *resid, const void *y,
                                 void *resid_out, void *norm_out, cudaStream_t stream) {
    if (r.T == 0) return cudaSuccess;
    ForwardArgs a = forward_args(r, resid, resid_out, norm_out);
    a.y = y;
    return forward<false>(r, a, stream);
}

cudaError_t launch_combine_residual_norm(const ResidualNorm &r, const void *y_perm,
                                         const int *row_of, const float *topk_w, int k,
                                         int64_t rows_alloc, const void *resid, void *y_out,
                                         void *resid_out, void *norm_out, int *status,
                                         cudaStream_t stream) {
    if (r.T == 0) return cudaSuccess;
    ForwardArgs a = forward_args(r, resid, resid_out, norm_out);
    a.y = y_perm;
    a.y_out = y_out;
    a.row_of = row_of;
    a.topk_w = topk_w;
    a.k = k;
    a.rows_alloc = rows_alloc;
    a.status = status;
    return forward<true>(r, a, stream);
}

int residual_parts(int T, int D) { return std::min(T, D <= 1024 ? 1216 : D <= 4096 ? 608 : 304); }

cudaError_t launch_residual_norm_backward(const ResidualNorm &r, const void *s, const void *y,
                                          const void *dresid_out, const void *dnorm_out,
                                          void *dresid, void *dy, float *dpost, void *dgate,
                                          float *dpre, float *part, cudaStream_t stream) {
    cudaError_t err;
    float *sums[3] = {dpre, dpost, r.gate_kind == GATE_CHANNEL ? (float *)dgate : nullptr};
    const int parts = residual_parts(r.T, r.D);
    if (r.T > 0) {
        BackwardArgs a = {};
        a.s = s;
        a.y = y;
        a.post = r.post;
        a.gate = r.gate;
        a.pre = r.pre;
        a.ds_out = dresid_out;
        a.dn = dnorm_out;
        a.dresid = dresid;
        a.dy = dy;
        a.dgate = dgate;
        a.part = part;
        a.drop = make_drop(r);
        a.eps = r.eps;
        a.res_scale = r.res_scale;
        a.branch_scale = r.branch_scale;
        a.T = r.T;
        a.D = r.D;
        a.gate_kind = r.gate_kind;
        int threads, nv;
        row_shape(r.D / 8, &threads, &nv);
        auto kernel = r.is_bf16 ? (nv == 1   ? residual_norm_backward_kernel<true, 1>
                                   : nv == 2 ? residual_norm_backward_kernel<true, 2>
                                             : residual_norm_backward_kernel<true, 4>)
                                : (nv == 1   ? residual_norm_backward_kernel<false, 1>
                                   : nv == 2 ? residual_norm_backward_kernel<false, 2>
                                             : residual_norm_backward_kernel<false, 4>);
        err = launch_pdl(kernel, dim3(parts), dim3(threads), 0, stream, a);
        if (err != cudaSuccess) return err;
        count_launch();
    }
    if (!sums[0] && !sums[1] && !sums[2]) return cudaSuccess;
    FinishArgs f = {};
    f.part = part;
    for (int i = 0; i < 3; ++i) f.out[i] = sums[i];
    f.parts = parts;  // none without rows: the sums are zero
    f.D = r.D;
    err = launch_pdl(residual_finish_kernel, dim3((r.D + FIN_COLS - 1) / FIN_COLS, 3),
                     dim3(FIN_COLS, FIN_ROWS), 0, stream, f);
    if (err == cudaSuccess) count_launch();
    return err;
}

}  // namespace moe
