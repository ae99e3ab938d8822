// The norms around a block, fused with its gate, dropout and residual sum.
//
// Per token (row of D values), with resid r, branch output y:
//   v = y                                    without a post gain,
//   v = y rsqrt(mean(y^2) + eps) post        with one;
//   s = res_scale r + branch_scale gate keep v          (the new residual)
//   n = s rsqrt(mean(s^2) + eps) pre                    (the next block's input)
// keep is 0 or 1 / (1 - p) from a counter-based generator (philox below), so
// no mask is stored: forward and gradient derive it from (seed, offset).
// All arithmetic is fp32; s and n are rounded once each, and n is the norm of
// the unrounded s.
//
// Every element is touched a fixed few times, so the passes are bound by HBM:
// forward 4 T D elements (r, y in; s, n out), gradient 6 (s, y, ds, dn in; dr,
// dy out), and close behind by instructions: at 2 bytes an element the copy rate
// leaves about 20 per element and warp lane.  A row's values stay on the SM
// between its sums, and the next row is on its way meanwhile.  Measured on GB300
// (bf16, of the copy rate; inputs larger than L2): 16384 x 4096 forward 86.4-87.5 us
// (91%), its gradient 134 (88%), gradient of 8192 x 7168 115.8 (90%); dropout's
// generator adds 12 us to 45 at 16384 x 2048; fp32 8192 x 2048 forward 47 (84%),
// gradient 74 (80%).  Behind the combine (16384 x 2048, 6 rows a token) 119 us
// (83%): a row's loads wait for its places, and more of them in flight per thread
// or in a shared ring measured slower (8192 x 4096, 4 rows: 101 us, a ring 134).
// The order of a row's sums and products goes by the kernel and its threads, so
// by T and D: among more rows the same row may differ in its last bits.
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
        float *q = static_cast<float *>(p) + 8 * vec;
        if ((reinterpret_cast<uintptr_t>(q) & 31) == 0) {  // a whole sector at once
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "f"(f[0]),
                         "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                         : "memory");
        } else {
            reinterpret_cast<float4 *>(q)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(q)[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
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

// ---------------------------------------------------------------------
// arithmetic on pairs
// ---------------------------------------------------------------------
// Pairs of fp32, added and multiplied two at a time.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 parts(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 both(float x) { return pair(x, x); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float sum2(f2 v) {
    const float2 p = parts(v);
    return p.x + p.y;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const Pack<BF16> &p, f2 (&f)[4]) {
    float v[8];
    unpack8<BF16>(p, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(v[2 * i], v[2 * i + 1]);
}
template <bool BF16>
__device__ __forceinline__ void store8(void *p, size_t vec, const f2 (&f)[4]) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = parts(f[i]);
        v[2 * i] = q.x;
        v[2 * i + 1] = q.y;
    }
    store8<BF16>(p, vec, v);
}

__device__ __forceinline__ void put8(float *shared, const f2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float2 *>(shared)[i] = parts(f[i]);
}

// Bit e: element e of a vector stays: half word e of the vector's four words, low half first.
__device__ __forceinline__ uint32_t keep_bits(uint64_t vec, uint32_t cut, uint64_t seed,
                                              uint64_t offset) {
    const uint4 w = philox(vec, offset, seed);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bits |= ((u[i] & 0xffffu) >= cut ? 1u : 0u) << (2 * i);
        bits |= ((u[i] >> 16) >= cut ? 1u : 0u) << (2 * i + 1);
    }
    return bits;
}
__device__ __forceinline__ f2 kept(f2 v, uint32_t bits, int i) {
    const float2 p = parts(v);
    return pair(bits >> (2 * i) & 1u ? p.x : 0.f, bits >> (2 * i + 1) & 1u ? p.y : 0.f);
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
// a thread's own columns of the next rows, in shared memory
// ---------------------------------------------------------------------
// Thread `mine` of the `across` that share a row copies vectors mine + i across
// (i < NV) of up to 5 arrays with cp.async and alone reads them back (fp32: a warp
// copies for its lanes), so that the next rows are in flight while one is worked
// on and nothing has to be waited for but one's own copies.  [depth][array][NV]
// planes, in each a vector of 16 or 32 bytes for every thread of the CTA.  Of an
// fp32 vector's two 16-byte pieces every other four threads have the second one
// first, so that eight threads' reads lie in different banks; both stay within
// the vector's 32 bytes, or a copy would fetch its sector twice.
template <bool BF16, int NV> struct Ring {
    static constexpr int EB = BF16 ? 16 : 32;  // bytes of a vector
    char *own;
    uint32_t plane, stage_bytes;
    int V, mine, across, depth;

    __device__ __forceinline__ Ring(char *smem, int V_, int mine_, int across_, int depth_, int arrays)
        : own(smem + threadIdx.x * EB), plane(blockDim.x * EB), stage_bytes(arrays * NV * plane), V(V_),
          mine(mine_), across(across_), depth(depth_) {
#pragma unroll
        for (int i = 0; i < NV; ++i)  // columns past the row's end read zeros
            if (mine + i * across >= V)
                for (int k = 0; k < depth * arrays; ++k)
#pragma unroll
                    for (int h = 0; h < EB / 16; ++h)
                        *reinterpret_cast<uint4 *>(own + (k * NV + i) * plane + 16 * h) =
                            make_uint4(0, 0, 0, 0);
    }
    // where thread `t` has piece h of its fp32 vector, within the vector
    __device__ __forceinline__ static int swapped(int t, int h) { return (h ^ (t >> 2 & 1)) * 16; }
    __device__ __forceinline__ void copy(const void *array, int k, size_t base, int stage) {
        const uint32_t at = smem_u32(own) + stage * stage_bytes + k * NV * plane;
        const char *src = static_cast<const char *>(array) + base * EB;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (BF16) {
                const int v = mine + i * across;
                if (v < V) copy_piece(at + i * plane, src + (size_t)v * 16);
            } else {
                // A warp's 32 vectors are 64 pieces in a row: a lane takes pieces
                // lane and lane + 32, so that each copy reads 512 bytes on end,
                // and puts them where the vector's own lane looks.
                const int lane = threadIdx.x & 31;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int q = 32 * h + lane, to = q >> 1, v = mine - lane + i * across + to;
                    if (v < V)
                        copy_piece(at + i * plane + (to - lane) * 32 + swapped(to, q & 1),
                                   src + (size_t)v * 32 + 16 * (q & 1));
                }
            }
        }
    }
    __device__ __forceinline__ static void copy_piece(uint32_t dst, const char *src) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    }
    __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // the oldest of `depth` (2 or 3) committed rows is there
    __device__ __forceinline__ void wait() {
        switch (depth) {
        case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        }
        if (!BF16) __syncwarp();
    }
    // before a slot that the warp has read is copied into again
    __device__ __forceinline__ void reuse() {
        if (!BF16) __syncwarp();
    }
    __device__ __forceinline__ void drain() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
    __device__ __forceinline__ Pack<BF16> take(int k, int i, int stage) const {
        const char *p = own + stage * stage_bytes + (k * NV + i) * plane;
        Pack<BF16> r;
        if constexpr (BF16) {
            r.a = *reinterpret_cast<const uint4 *>(p);
        } else {
            r.a = *reinterpret_cast<const uint4 *>(p + swapped(threadIdx.x, 0));
            r.b = *reinterpret_cast<const uint4 *>(p + swapped(threadIdx.x, 1));
        }
        return r;
    }
};

// ---------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------
struct ForwardArgs {
    const void *resid, *y, *post, *gate, *pre;
    void *y_out, *resid_out, *norm_out;
    Drop drop;
    float eps, res_scale, branch_scale;
    int T, D, gate_kind;
    int depth, in_ring;  // rows and arrays of the ring kernel's
    // the combine in front (COMBINE): y[t] = sum_j topk_w[t, j] y_perm[row_of[t, j]]
    const int *row_of;
    const float *topk_w;
    int k;
    long long rows_alloc;
    int *status;
};

// 8 values of an expert's row: fp16 with bf16 layers, else fp32.
template <bool BF16>
__device__ __forceinline__ Pack<BF16> expert_load8(const void *y_perm, size_t vec) {
    Pack<BF16> r;
    const uint4 *p = static_cast<const uint4 *>(y_perm) + (BF16 ? vec : 2 * vec);
    r.a = __ldcs(p);
    if constexpr (!BF16) r.b = __ldcs(p + 1);
    return r;
}
template <bool BF16>
__device__ __forceinline__ void expert_unpack8(const Pack<BF16> &q, float (&f)[8]) {
    if constexpr (BF16) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&q.a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(h[i]);
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    } else {
        unpack8<false>(q, f);
    }
}

// One row per CTA at a time, straight from global memory: few rows, the widest
// ones, and behind the combine.
// NV vectors of 8 per thread: vector tid + i blockDim of the row.
template <bool BF16, int NV, bool COMBINE>
__global__ void __launch_bounds__(1024)
residual_norm_row_kernel(const ForwardArgs a) {
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
    int row = -1;
    float w = 0.f;
    auto read_places = [&](long long t) {
        if (t >= a.T) return;
        row = a.row_of[t * a.k + tid];
        w = a.topk_w[t * a.k + tid];
    };
    if (COMBINE && tid < a.k) read_places(blockIdx.x);
    int turn = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t base = (size_t)t * V;
        if constexpr (COMBINE) {
            __syncthreads();  // the row before is done with s_row
            if (tid < a.k) {
                if (row < -1 || (long long)row >= a.rows_alloc) {
                    raise_flag(a.status, FLAG_BAD_ROUTING);
                    row = -1;
                }
                s_row[tid] = row;
                s_w[tid] = w;
                read_places(t + gridDim.x);  // of the next row: there when this one is done
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
            if (!COMBINE && branch) unpack8<BF16>(load8<BF16>(a.y, base + v), y[i]);
        }
        if constexpr (COMBINE) {
            for (int j = 0; j < a.k; ++j) {
                if (s_row[j] < 0) continue;
                const float wj = s_w[j];
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = tid + i * blockDim.x;
                    if (v >= V) continue;
                    float f[8];
                    expert_unpack8<BF16>(expert_load8<BF16>(a.y, (size_t)s_row[j] * V + v), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[i][e] = fmaf(wj, f[e], y[i][e]);
                }
            }
            if (a.y_out) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (tid + i * blockDim.x < V) store8<BF16>(a.y_out, base + tid + i * blockDim.x, y[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[0] = fmaf(y[i][e], y[i][e], sum[0]);
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
                if (a.drop.cut) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[i][e] *= a.drop.scale;
                }
                if (a.gate_kind == GATE_CHANNEL || a.gate_kind == GATE_ELEMENT) {
                    unpack8<BF16>(load8<BF16>(a.gate, a.gate_kind == GATE_CHANNEL ? v : base + v), g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[i][e] *= g[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) y[i][e] = a.branch_scale * (gt * y[i][e]);
                if (a.drop.cut) {  // last: nothing of a dropped element, be it infinite
                    const uint32_t bits = keep_bits(base + v, a.drop.cut, seed, offset);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[i][e] = bits >> e & 1u ? y[i][e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) s[i][e] = fmaf(a.res_scale, s[i][e], y[i][e]);
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

// Many rows: a row per CTA (WARP: per warp, narrow rows) at a time, the next ones
// in a Ring.  FULL: a branch and the next norm, no gate for every element.
template <bool BF16, int NV, bool WARP, bool FULL>
__global__ void __launch_bounds__(256, NV == 4 && WARP ? 1 : 2)
residual_norm_ring_kernel(const ForwardArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ float s_sum[2][32];
    griddep_launch_dependents();
    griddep_wait();
    const int V = a.D / 8, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mine = WARP ? lane : tid, across = WARP ? 32 : blockDim.x;
    const int unit = WARP ? blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
    const int units = WARP ? gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const float inv_d = 1.f / (float)a.D;
    const bool branch = FULL || a.y, elem = !FULL && a.gate_kind == GATE_ELEMENT;
    const bool has_pre = FULL || a.pre, drops = a.drop.cut > 0;
    uint64_t seed = 0, offset = 0;
    if (drops) {
        seed = (uint64_t)a.drop.rng[0];
        offset = (uint64_t)a.drop.rng[1];
    }
    Pack<BF16> pre[NV];
    f2 coef[NV][4];  // branch_scale, the dropout's factor, post, a channel's gate
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = mine + i * across;
        pre[i] = Pack<BF16>{};
#pragma unroll
        for (int e = 0; e < 4; ++e) coef[i][e] = both(a.branch_scale * (drops ? a.drop.scale : 1.f));
        if (v >= V) continue;
        f2 f[4];
        if (has_pre) pre[i] = load8<BF16>(a.pre, v);
        if (a.post) {
            unpack8<BF16>(load8<BF16>(a.post, v), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) coef[i][e] = mul2(coef[i][e], f[e]);
        }
        if (a.gate_kind == GATE_CHANNEL) {
            unpack8<BF16>(load8<BF16>(a.gate, v), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) coef[i][e] = mul2(coef[i][e], f[e]);
        }
    }
    Ring<BF16, NV> ring(smem, V, mine, across, a.depth, a.in_ring);
    auto copy_row = [&](long long t, int stage) {
        if (t < a.T) {
            const size_t base = (size_t)t * V;
            ring.copy(a.resid, 0, base, stage);
            if (branch) ring.copy(a.y, 1, base, stage);
            if (elem) ring.copy(a.gate, 2, base, stage);
        }
        ring.commit();
    };
    int turn = 0, stage = 0;
    auto row_sum = [&](float x) {
        float v[1] = {x};
        if (WARP) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        } else {
            block_sum<1>(v, s_sum[turn]);
            turn ^= 1;
        }
        return v[0];
    };
    for (int i = 0; i < a.depth - 1; ++i) copy_row(unit + (long long)i * units, i);
    for (long long t = unit; t < a.T; t += units) {
        ring.reuse();
        copy_row(t + (long long)(a.depth - 1) * units, stage == 0 ? a.depth - 1 : stage - 1);
        ring.wait();
        const size_t base = (size_t)t * V;
        f2 s[NV][4];
        f2 sum;
        if (branch) {
            float r1 = a.gate_kind == GATE_TOKEN ? static_cast<const float *>(a.gate)[t] : 1.f;
            f2 y[NV][4];
#pragma unroll
            for (int i = 0; i < NV; ++i) unpack8<BF16>(ring.take(1, i, stage), y[i]);
            if (a.post) {
                sum = both(0.f);
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum = fma2(y[i][e], y[i][e], sum);
                r1 *= rsqrtf(fmaf(row_sum(sum2(sum)), inv_d, a.eps));
            }
            const f2 r1_2 = both(r1), res_2 = both(a.res_scale);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                unpack8<BF16>(ring.take(0, i, stage), s[i]);
                uint32_t bits = 0xffu;
                if (drops) bits = keep_bits(base + mine + i * across, a.drop.cut, seed, offset);
                f2 ge[4];
                if (elem) unpack8<BF16>(ring.take(2, i, stage), ge);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f2 v = mul2(mul2(y[i][e], r1_2), coef[i][e]);
                    if (elem) v = mul2(v, ge[e]);
                    if (drops) v = kept(v, bits, e);
                    s[i][e] = fma2(s[i][e], res_2, v);
                }
                if (mine + i * across < V) store8<BF16>(a.resid_out, base + mine + i * across, s[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) unpack8<BF16>(ring.take(0, i, stage), s[i]);
        }
        if (has_pre) {
            sum = both(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum = fma2(s[i][e], s[i][e], sum);
            const f2 r2_2 = both(rsqrtf(fmaf(row_sum(sum2(sum)), inv_d, a.eps)));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                f2 w[4];
                unpack8<BF16>(pre[i], w);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = mul2(mul2(s[i][e], r2_2), w[e]);
                if (mine + i * across < V) store8<BF16>(a.norm_out, base + mine + i * across, w);
            }
        }
        if (++stage == a.depth) stage = 0;
    }
    ring.drain();
}

// ---------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------
// Eight sums over a warp in nine exchanges: lanes trade halves of what they have
// until each holds one sum, lane 4 i .. 4 i + 3 the i-th.
__device__ __forceinline__ float warp_sums(float (&v)[8]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = 4, bit = 16; half > 0; half >>= 1, bit >>= 1) {
        const bool high = lane & bit;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float give = high ? v[i] : v[i + half], take = high ? v[i + half] : v[i];
            v[i] = take + __shfl_xor_sync(0xffffffffu, give, bit);
        }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// The same over the CTA (at most 32 warps; one barrier, `slot` as in block_sum);
// every thread gets the sums.
template <bool WARP>
__device__ __forceinline__ void row_sums(float (&v)[8], float *slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    float sum = warp_sums(v);
    if (!WARP) {
        if ((lane & 3) == 0) slot[(lane >> 2) * 32 + warp] = sum;
        __syncthreads();
        sum = 0.f;
        for (int w = lane & 3; w < nwarps; w += 4) sum += slot[(lane >> 2) * 32 + w];
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xffffffffu, sum, 4 * i);
}

struct BackwardArgs {
    const void *s, *y, *post, *gate, *pre, *ds_out, *dn;
    void *dresid, *dy, *dgate;
    float *part;  // [2][gridDim.x][D]: this CTA's column sums P and G
    Drop drop;
    float eps, res_scale, branch_scale;
    int T, D, gate_kind, depth;
    int in_ring;  // arrays there: 4, or 5 with a gate for every element
};

// With r1, r2 the rows' rsqrt factors and gp = dn pre:
//   ds = ds_out + r2 gp - c s r2,  c = r2^2 mean(gp s)
//   u = branch_scale keep ds;  dgate = u v;  dv = gate u
//   dy = r1 (dv post - y r1^2 mean(dv post y))
// ds is linear in two row sums that are not known yet, so with
// q = branch_scale keep post gate y,
//   sum(ds q) = sum(ds_out q) + r2 sum(gp q) - c r2 sum(s q)
// and every sum of the row comes out of ONE reduction.  (A token's gate is left
// out of q and multiplied in behind.)  The column sums are two:
//   P = sum dn s r2 = dpre,   G = sum keep ds y r1 (times a gate that is not the
//   channel's);  dpost = branch_scale gate G and dgate = branch_scale post G.
//
// A row per CTA (WARP: per warp, narrow rows), rows over the grid, in a Ring from
// which each thread reads its columns twice, before and behind the reduction
// (registers are short).  Rows too wide for two in shared memory are read from global memory
// instead, the second time from L2 (RING false: fp32 from D = 6664, or 5640 with a
// gate for every element, and all from 8200).  One CTA per SM, nothing copied
// ahead and registers spilled: 4096 x 7168 fp32 298 us (floor 104), 4096 x 12288
// bf16 289 (89), 2048 x 24576 bf16 537 (89).
//
// The kernel is as much bound by instructions as by bytes (per vector of 8 about
// 100 to unpack five operands twice, 80 of arithmetic two values at a time), so
// what is usual is known when it is compiled: FULL has both gradients, both norms'
// operands and no gate of its own for every element; DROP is dropout.  The rest
// asks as it goes.
template <bool BF16, int NV, bool WARP, bool FULL, bool DROP, bool RING>
__global__ void __launch_bounds__(WARP ? 256 : NV == 1 ? 256 : 512, NV == 1 ? 2 : 1)
residual_norm_backward_kernel(const BackwardArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ float s_sum[2][8 * 32];
    griddep_launch_dependents();
    griddep_wait();
    const int V = a.D / 8, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mine = WARP ? lane : tid, across = WARP ? 32 : blockDim.x;
    const int unit = WARP ? blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
    const int units = WARP ? gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const float inv_d = 1.f / (float)a.D;
    const bool branch = FULL || a.y, elem = !FULL && a.gate_kind == GATE_ELEMENT;
    const bool drops = FULL ? DROP : a.drop.cut > 0, has_pre = FULL || a.pre;
    const float dscale = drops ? a.drop.scale : 1.f;
    uint64_t seed = 0, offset = 0;
    if (drops) {
        seed = (uint64_t)a.drop.rng[0];
        offset = (uint64_t)a.drop.rng[1];
    }
    // what a column multiplies by: coef = branch_scale keep post gate (of a channel)
    Pack<BF16> pre[NV];
    f2 coef[NV][4], P[NV][4], G[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = mine + i * across;
        pre[i] = Pack<BF16>{};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            coef[i][e] = both(a.branch_scale * dscale);
            P[i][e] = G[i][e] = both(0.f);
        }
        if (v >= V) continue;
        f2 f[4];
        if (has_pre) pre[i] = load8<BF16>(a.pre, v);
        if (a.post) {
            unpack8<BF16>(load8<BF16>(a.post, v), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) coef[i][e] = mul2(coef[i][e], f[e]);
        }
        if (a.gate_kind == GATE_CHANNEL) {
            unpack8<BF16>(load8<BF16>(a.gate, v), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) coef[i][e] = mul2(coef[i][e], f[e]);
        }
    }

    // without the next norm ds is ds_out: s is left out, whatever it holds
    const void *arrays[5] = {has_pre ? a.s : nullptr, a.ds_out, a.dn, a.y, elem ? a.gate : nullptr};
    auto has = [&](int k) { return FULL ? k < 4 : arrays[k] != nullptr; };
    Ring<BF16, NV> ring(smem, V, mine, across, RING ? a.depth : 0, a.in_ring);
    auto copy_row = [&](long long t, int stage) {
        if (!RING) return;
        if (t < a.T) {
#pragma unroll
            for (int k = 0; k < 5; ++k)
                if (has(k)) ring.copy(arrays[k], k, (size_t)t * V, stage);
        }
        ring.commit();
    };
    auto take = [&](int k, int i, int stage, size_t base) {
        const Pack<BF16> none = {};
        if (!has(k)) return none;
        if (RING) return ring.take(k, i, stage);
        return mine + i * across < V ? load8<BF16>(arrays[k], base + mine + i * across) : none;
    };
    for (int i = 0; i < a.depth - 1; ++i) copy_row(unit + (long long)i * units, i);

    int turn = 0, stage = 0;
    for (long long row = unit; row < a.T; row += units, turn ^= 1) {
        const int t = (int)row;
        const int last = stage == 0 ? a.depth - 1 : stage - 1;  // read a row ago
        if (RING) ring.reuse();
        copy_row(t + (long long)(a.depth - 1) * units, last);
        if (RING) ring.wait();
        const size_t base = (size_t)t * V;
        const float gt = a.gate_kind == GATE_TOKEN ? static_cast<const float *>(a.gate)[t] : 1.f;
        uint32_t bits[NV];
        f2 m[6];
#pragma unroll
        for (int n = 0; n < 6; ++n) m[n] = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            bits[i] = 0xffu;
            if (drops) bits[i] = keep_bits(base + mine + i * across, a.drop.cut, seed, offset);
            f2 s[4], d[4], n[4], y[4], w[4];
            unpack8<BF16>(take(0, i, stage, base), s);
            unpack8<BF16>(take(1, i, stage, base), d);
            unpack8<BF16>(take(2, i, stage, base), n);
            unpack8<BF16>(take(3, i, stage, base), y);
            unpack8<BF16>(pre[i], w);
            if (elem) {
                f2 ge[4];
                unpack8<BF16>(take(4, i, stage, base), ge);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f2 y2 = y[e];
                    m[2] = fma2(y2, y2, m[2]);
                    y[e] = mul2(y2, ge[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 gp = mul2(n[e], w[e]);
                f2 q = mul2(y[e], coef[i][e]);
                if (drops) q = kept(q, bits[i], e);
                m[0] = fma2(s[e], s[e], m[0]);
                m[1] = fma2(gp, s[e], m[1]);
                if (!elem) m[2] = fma2(y[e], y[e], m[2]);
                m[3] = fma2(d[e], q, m[3]);
                m[4] = fma2(gp, q, m[4]);
                m[5] = fma2(s[e], q, m[5]);
            }
        }
        float sum[8] = {sum2(m[0]), sum2(m[1]), sum2(m[2]), sum2(m[3]), sum2(m[4]), sum2(m[5]), 0.f, 0.f};
        row_sums<WARP>(sum, s_sum[turn]);
        const float r2 = has_pre ? rsqrtf(fmaf(sum[0], inv_d, a.eps)) : 0.f;
        // r1 and r2 multiply what they bring near one, a step at a time: their squares
        // and cubes leave the range of fp32 long before a row does
        const float c = r2 * (r2 * (sum[1] * inv_d));  // of s r2
        const float r1 = a.post ? rsqrtf(fmaf(sum[2], inv_d, a.eps)) : 1.f;
        const float dot = sum[3] + r2 * sum[4] - c * (r2 * sum[5]);  // sum(ds q)
        const float c1 = a.post ? r1 * (r1 * (dot * inv_d)) : 0.f;   // of gate y r1
        if (a.gate_kind == GATE_TOKEN && mine == 0) static_cast<float *>(a.dgate)[t] = r1 * dot;
        asm volatile("" ::: "memory");  // the row is read again, not kept: registers are short
        const f2 r2_2 = both(r2), c_2 = both(-c), res_2 = both(branch ? a.res_scale : 1.f);
        const f2 r1_2 = both(r1), g_2 = both(r1 * gt), c1_2 = both(-c1);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = mine + i * across;
            if (v >= V) continue;
            f2 s[4], d[4], n[4], y[4], w[4], ge[4];
            unpack8<BF16>(take(0, i, stage, base), s);
            unpack8<BF16>(take(1, i, stage, base), d);
            unpack8<BF16>(take(2, i, stage, base), n);
            unpack8<BF16>(take(3, i, stage, base), y);
            unpack8<BF16>(pre[i], w);
            if (elem) unpack8<BF16>(take(4, i, stage, base), ge);
            if (drops && !a.post) {  // a dropped y may be infinite (under a norm the row is lost then)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = kept(y[e], bits[i], e);
            }
            if (elem && drops) {  // and so may its gate
#pragma unroll
                for (int e = 0; e < 4; ++e) ge[e] = kept(ge[e], bits[i], e);
            }
            f2 dg[4], yr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 sr = mul2(s[e], r2_2);
                yr[e] = mul2(y[e], g_2);
                const f2 ds = fma2(sr, c_2, fma2(mul2(n[e], w[e]), r2_2, d[e]));
                P[i][e] = fma2(n[e], sr, P[i][e]);
                f2 k = drops ? kept(ds, bits[i], e) : ds;
                if (elem) {
                    dg[e] = mul2(mul2(k, coef[i][e]), mul2(y[e], r1_2));
                    k = mul2(k, ge[e]);
                }
                G[i][e] = fma2(k, yr[e], G[i][e]);
                d[e] = mul2(ds, res_2);
                y[e] = mul2(mul2(k, coef[i][e]), g_2);
            }
            if (a.post) {  // no mean without a norm, whatever y holds
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = fma2(yr[e], c1_2, y[e]);
            }
            store8<BF16>(a.dresid, base + v, d);
            if (branch) store8<BF16>(a.dy, base + v, y);
            if (elem) store8<BF16>(a.dgate, base + v, dg);
        }
        if (++stage == a.depth) stage = 0;
    }
    ring.drain();

    // The CTA's column sums.  A channel's gate takes the token's gate for one:
    // G holds neither.
    if (!a.pre && !a.post && a.gate_kind != GATE_CHANNEL) return;
    float *part = a.part + (size_t)blockIdx.x * a.D;
    const size_t to_G = (size_t)gridDim.x * a.D;
    if (!WARP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = mine + i * across;
            if (v >= V) continue;
            store8<false>(part, v, P[i]);
            store8<false>(part + to_G, v, G[i]);
        }
        return;
    }
    // the warps' sums through the ring, P then G
    const int nwarps = blockDim.x >> 5;
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (mine + i * across < V)
                put8(sums + (size_t)warp * a.D + 8 * (mine + i * across), which ? G[i] : P[i]);
        __syncthreads();
        for (int d = tid; d < a.D; d += blockDim.x) {
            float x = 0.f;
            for (int w = 0; w < nwarps; ++w) x += sums[(size_t)w * a.D + d];
            part[which * to_G + d] = x;
        }
    }
}

// dpre, dpost and a channel gate's gradient from the CTAs' parts, added in a
// fixed order.  blockIdx.y: P or G.
struct FinishArgs {
    const float *part;
    const void *post, *gate;  // the other factor of dgate and dpost, or null
    float *dpre, *dpost, *dgate;
    float scale;  // branch_scale and the dropout's factor
    int parts, D, is_bf16;
};

__device__ __forceinline__ float factor_at(const void *p, int c, int is_bf16) {
    if (!p) return 1.f;
    return is_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[c])
                   : static_cast<const float *>(p)[c];
}

constexpr int FIN_COLS = 32, FIN_ROWS = 32;
__global__ void __launch_bounds__(FIN_COLS *FIN_ROWS)
residual_finish_kernel(const FinishArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float s[FIN_ROWS][FIN_COLS];
    const bool is_G = blockIdx.y;
    if (is_G ? !a.dpost && !a.dgate : !a.dpre) return;
    const int c = blockIdx.x * FIN_COLS + threadIdx.x, r = threadIdx.y;
    const float *p = a.part + (is_G ? (size_t)a.parts * a.D : 0);
    float sum = 0.f;
    if (c < a.D)
#pragma unroll 5
        for (int i = r; i < a.parts; i += FIN_ROWS) sum += p[(size_t)i * a.D + c];
    s[r][threadIdx.x] = sum;
    __syncthreads();
    if (r == 0 && c < a.D) {
#pragma unroll
        for (int i = 1; i < FIN_ROWS; ++i) sum += s[i][threadIdx.x];
        if (!is_G) {
            a.dpre[c] = sum;
        } else {
            sum *= a.scale;
            if (a.dpost) a.dpost[c] = sum * factor_at(a.gate, c, a.is_bf16);
            if (a.dgate) a.dgate[c] = sum * factor_at(a.post, c, a.is_bf16);
        }
    }
}

// Bytes of one row's slot of a Ring.
size_t ring_bytes(int arrays, int nv, int is_bf16, int threads) {
    return (size_t)arrays * nv * threads * (is_bf16 ? 16 : 32);
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
cudaError_t forward_rows(const ResidualNorm &r, const ForwardArgs &a, cudaStream_t stream) {
    int threads, nv;
    const int V = r.D / 8;
    row_shape(V, &threads, &nv);
    auto kernel = r.is_bf16 ? (nv == 1   ? residual_norm_row_kernel<true, 1, COMBINE>
                               : nv == 2 ? residual_norm_row_kernel<true, 2, COMBINE>
                                         : residual_norm_row_kernel<true, 4, COMBINE>)
                            : (nv == 1   ? residual_norm_row_kernel<false, 1, COMBINE>
                               : nv == 2 ? residual_norm_row_kernel<false, 2, COMBINE>
                                         : residual_norm_row_kernel<false, 4, COMBINE>);
    const int grid = std::min(r.T, std::max(1, sm_count()) * std::max(1, 2048 / threads));
    const cudaError_t err = launch_pdl(kernel, dim3(grid), dim3(threads), 0, stream, a);
    if (err == cudaSuccess) count_launch();
    return err;
}

cudaError_t forward(const ResidualNorm &r, ForwardArgs &a, cudaStream_t stream) {
    const int V = r.D / 8;
    const bool warp = V <= 128;
    // What a row costs besides its vectors (two reductions, its copies' addresses)
    // is paid by every warp, so few warps take several vectors each (16384 x 4096:
    // one vector 95.8 us, two 86.5), and two rows in the ring are in flight enough
    // (two 86.5, three 89.9, four 93.0).
    const int nv = warp ? (V <= 32 ? 1 : V <= 64 ? 2 : 4) : V <= 512 ? 2 : 4;
    const int threads = warp ? 256 : ((V + nv - 1) / nv + 31) / 32 * 32;
    a.in_ring = r.gate_kind == GATE_ELEMENT ? 3 : 2;
    const size_t stage = ring_bytes(a.in_ring, nv, r.is_bf16, threads);
    int per_sm = warp ? (nv == 4 ? 1 : 2) : std::min(8, 512 / threads);
    while (per_sm > 1 && 2 * stage * per_sm > 220 * 1024) --per_sm;
    a.depth = 2 * stage * per_sm > 220 * 1024 ? 1 : 2;
    const int at_once = sm_count() * per_sm * (warp ? 8 : 1);
    // one row a CTA leaves nothing to copy ahead: then, and for the widest rows,
    // straight from global memory
    if (V > 1024 || a.depth < 2 || r.T <= at_once) return forward_rows<false>(r, a, stream);
    using Kernel = void (*)(ForwardArgs);
#define MOE_RINGS(BF16, FULL)                                                                   \
    {residual_norm_ring_kernel<BF16, 1, true, FULL>, residual_norm_ring_kernel<BF16, 2, true, FULL>, \
     residual_norm_ring_kernel<BF16, 4, true, FULL>, residual_norm_ring_kernel<BF16, 2, false, FULL>, \
     residual_norm_ring_kernel<BF16, 4, false, FULL>}
    static const Kernel kernels[2][2][5] = {{MOE_RINGS(false, false), MOE_RINGS(false, true)},
                                            {MOE_RINGS(true, false), MOE_RINGS(true, true)}};
#undef MOE_RINGS
    const bool is_full = a.y && a.pre && r.gate_kind != GATE_ELEMENT;
    const int which = warp ? (nv == 4 ? 2 : nv - 1) : (nv == 4 ? 4 : 3);
    const Kernel kernel = kernels[r.is_bf16 ? 1 : 0][is_full ? 1 : 0][which];
    cudaError_t err = ensure_smem((const void *)kernel, stage * a.depth);
    if (err != cudaSuccess) return err;
    err = launch_pdl(kernel, dim3(sm_count() * per_sm), dim3(threads), stage * a.depth, stream, a);
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
    return forward(r, a, stream);
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
    return forward_rows<true>(r, a, stream);
}

// Shape of a gradient launch.
struct GradientShape {
    int nv, threads, depth, ctas, in_ring;
    bool warp, ring;
    size_t smem;
};

namespace {

constexpr int kMaxParts = 4 * 152;  // of the column sums: what a workspace has room for

// A row per warp up to 512 columns, else per CTA, with as few vectors a thread as
// 256 threads allow (4096 x 2048: one 24.7 us, two 27.1).  Two rows in the ring
// where a thread has two vectors, else three (16384 x 4096: 134.5 us with two, 147
// with three; 16384 x 2048: 73.8 and 70.5): more in flight than DRAM needs costs.
// With dropout a row's instructions bound it, and over many rows two vectors a
// thread share them (16384 x 2048: 86.1 us, one 100.8; 4096 rows: 34.5 and 32.0).
GradientShape gradient_shape(int T, int D, int is_bf16, int gate_kind, bool drops) {
    GradientShape g = {};
    const int V = D / 8;
    g.warp = V <= 64;
    g.nv = (g.warp ? V <= 32 : V <= (drops && T >= 8192 ? 192 : 256)) ? 1 : 2;
    g.threads = g.warp ? 256 : ((V + g.nv - 1) / g.nv + 31) / 32 * 32;
    g.in_ring = gate_kind == GATE_ELEMENT ? 5 : 4;
    const size_t stage = ring_bytes(g.in_ring, g.nv, is_bf16, g.threads);
    // CTAs per SM by their registers, fewer where two rows each are too much
    int per_sm = g.warp ? 3 - g.nv : std::max(1, std::min(4, 512 / g.threads));
    auto fit = [&] { return (int)std::min<size_t>(g.nv == 1 ? 3 : 2, (size_t)(220 * 1024 / per_sm) / stage); };
    while (per_sm > 1 && fit() < 2) --per_sm;
    g.depth = fit();
    g.ring = V <= 1024 && g.depth >= 2;
    g.smem = g.warp ? std::max(stage * g.depth, (size_t)8 * D * 4) : stage * g.depth;
    if (!g.ring) {
        g.nv = V <= 2048 ? 4 : 8;
        g.threads = ((V + g.nv - 1) / g.nv + 31) / 32 * 32;
        g.depth = 1;
        g.smem = 0;
        per_sm = 1;
    }
    const int rows = g.warp ? 8 : 1;  // at a time in a CTA
    g.ctas = std::min(T / rows + (T % rows != 0), std::min(sm_count() * per_sm, kMaxParts));
    return g;
}

}  // namespace

int residual_parts(int T) { return std::min(T, kMaxParts); }

cudaError_t launch_residual_norm_backward(const ResidualNorm &r, const void *s, const void *y,
                                          const void *dresid_out, const void *dnorm_out,
                                          void *dresid, void *dy, float *dpost, void *dgate,
                                          float *dpre, float *part, cudaStream_t stream) {
    cudaError_t err;
    const GradientShape g = gradient_shape(r.T, r.D, r.is_bf16, r.gate_kind, r.drop_cut > 0);
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
        a.depth = g.depth;
        a.in_ring = g.in_ring;
        using Kernel = void (*)(BackwardArgs);
        // [type][a row per warp: 1, 2 vectors a lane; per CTA: 1, 2; without a ring: 4, 8]
#define MOE_RINGS(BF16, FULL, DROP)                                                             \
    residual_norm_backward_kernel<BF16, 1, true, FULL, DROP, true>,                               \
        residual_norm_backward_kernel<BF16, 2, true, FULL, DROP, true>,                           \
        residual_norm_backward_kernel<BF16, 1, false, FULL, DROP, true>,                          \
        residual_norm_backward_kernel<BF16, 2, false, FULL, DROP, true>
#define MOE_ANY(BF16)                                                                           \
    MOE_RINGS(BF16, false, false), residual_norm_backward_kernel<BF16, 4, false, false, false, false>, \
        residual_norm_backward_kernel<BF16, 8, false, false, false, false>
        static const Kernel any[2][6] = {{MOE_ANY(false)}, {MOE_ANY(true)}};
        static const Kernel full[2][2][4] = {{{MOE_RINGS(false, true, false)}, {MOE_RINGS(false, true, true)}},
                                             {{MOE_RINGS(true, true, false)}, {MOE_RINGS(true, true, true)}}};
#undef MOE_RINGS
#undef MOE_ANY
        const int which = g.warp ? g.nv - 1 : g.ring ? 1 + g.nv : g.nv == 4 ? 4 : 5;
        const bool is_full = g.ring && y && dresid_out && r.pre && r.gate_kind != GATE_ELEMENT;
        const Kernel kernel = is_full ? full[r.is_bf16 ? 1 : 0][r.drop_cut > 0 ? 1 : 0][which]
                                      : any[r.is_bf16 ? 1 : 0][which];
        if ((err = ensure_smem((const void *)kernel, g.smem)) != cudaSuccess) return err;
        err = launch_pdl(kernel, dim3(g.ctas), dim3(g.threads), g.smem, stream, a);
        if (err != cudaSuccess) return err;
        count_launch();
    }
    FinishArgs f = {};
    f.part = part;
    f.dpre = dpre;
    f.dpost = dpost;
    if (r.gate_kind == GATE_CHANNEL) {
        f.dgate = (float *)dgate;
        f.gate = r.gate;
    }
    f.post = r.post;
    if (!f.dpre && !f.dpost && !f.dgate) return cudaSuccess;
    f.scale = r.branch_scale * make_drop(r).scale;
    f.parts = g.ctas;  // none without rows: the sums are zero
    f.D = r.D;
    f.is_bf16 = r.is_bf16;
    err = launch_pdl(residual_finish_kernel, dim3((r.D + FIN_COLS - 1) / FIN_COLS, 2),
                     dim3(FIN_COLS, FIN_ROWS), 0, stream, f);
    if (err == cudaSuccess) count_launch();
    return err;
}

}  // namespace moe
