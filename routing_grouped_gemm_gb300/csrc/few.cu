// The whole layer for a few tokens, in one kernel.
//
//   key = x Wg^T + b, top-k and weights w;  h_j = SiLU(w1_e x) * (w3_e x);
//   out[t] = sum_j w_j (w2_e h_j),  e = the token's j-th expert.
//
// With T <= 32 tokens every weight of a chosen expert is used for a handful of
// rows, so the layer is bound by streaming the chosen experts' weights from HBM
// (3 D H values each), and by the latency of whatever stands before that stream.
// Launched as five steps, the steps' launches and tails cost about as much as
// the stream itself; here one CTA per SM runs all of them, with two barriers
// across the grid (cooperative launch):
//
//   route    expert rows of Wg over the CTAs, one dot product per token
//   -- barrier -- every CTA selects all tokens' experts for itself and sorts the
//            (token, slot) pairs by expert; at most 8 pairs of an expert form an
//            ENTRY, one pass over that expert's weights
//   GEMM1    tiles of 8 gate and 8 up rows of one entry over the CTAs -> h
//   -- barrier -- the loads of w2 begin before it: they do not depend on h
//   GEMM2    tiles of 16 rows of out; all (tile, entry, chunk of H) triples in
//            one line, cut into equal parts over the CTAs, so that the stream
//            ends everywhere at once.  A tile cut by that gets its parts' fp32
//            sums through memory, added by the CTA that comes last, in order.
//
// The 16 weight rows of a tile are the M side of mma.sync m16n8k16 and the
// entry's rows the N = 8 side: at 8 rows per weight the tensor pipe idles either
// way, and register accumulators need no TMEM round trip.  The CTA's 16 warps
// split k: of every 1 KB of a row a warp takes 64 bytes, and a lane copies its
// own 16 bytes of a row (the sum over k does not care which k meet in one
// instruction, as long as both operands agree) with cp.async into a ring that it
// alone reads back, so the stream needs no barrier but the sum over the warps at
// a tile's end, and the copies of the next tiles run through it.  (Bulk copies by
// a producer warp: each costs 55 ns to issue whatever its size, so 16 row pieces
// of 1 KB per stage reached 39% of the copy rate, of 4 KB 97% in long rows.)
// fp32 layers use the same tiles with fused multiply-adds.
//
// Rounding: keys, weights, both products' sums and the sum over experts are
// fp32; h is rounded to the layer's type once (as in moe_grouped_swiglu), out
// once.  Every sum has a fixed order for a given grid, so results do not change
// from run to run.
#include <algorithm>

#include <stdlib.h>
#include <string.h>

#include "common.cuh"
#include "launch.h"
#include "topk.cuh"

namespace moe {
namespace {

constexpr int FW_WARPS = 16;
constexpr int FW_THREADS = 32 * FW_WARPS;
constexpr int FW_STEP = 64;                    // bytes of a row that a warp takes at once
constexpr int FW_CHUNK = FW_STEP * FW_WARPS;   // and the CTA
constexpr int FW_M = 16;                       // weight rows per tile
constexpr int FW_N = 8;                        // rows of an entry
constexpr int FW_SLOT = 3 * 512;               // a warp's step in the ring: 8 + 8 weight rows, 8 rows

enum { FEW_ROUTE = 1, FEW_GEMM1 = 2, FEW_GEMM2 = 4, FEW_ALL = 7 };

struct FewParams {
    const void *x, *wg, *w1, *w3, *w2;
    const float *bias;
    void *out, *h;     // h: [T k][H] by the pair's place in the sorted order
    float *logits;     // [T][E]
    float *part;       // [gridDim.x][2][T][16]
    int *bars;         // [0], [1] the grid barriers, [2] CTAs done; zero between calls
    int *tile_count;   // [ceil(D / 16)] parts in; zero between calls
    int *status;
    int T, D, H, E, k, e_first, E_local, score, renorm, n_group, topk_group;
    int phases;
};

template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float round(float v) { return v; }
};
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};

// 16 bytes global -> shared, past L1; zeros when !in (src is not read then).
__device__ __forceinline__ void copy16(void *dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float dot_bf16x2(uint32_t a, uint32_t b, float c) {
    c = fmaf(__uint_as_float(a << 16), __uint_as_float(b << 16), c);
    return fmaf(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u), c);
}
template <typename T> __device__ __forceinline__ float dot16(uint4 a, uint4 b, float c);
template <> __device__ __forceinline__ float dot16<__nv_bfloat16>(uint4 a, uint4 b, float c) {
    c = dot_bf16x2(a.x, b.x, c);
    c = dot_bf16x2(a.y, b.y, c);
    c = dot_bf16x2(a.z, b.z, c);
    return dot_bf16x2(a.w, b.w, c);
}
template <> __device__ __forceinline__ float dot16<float>(uint4 a, uint4 b, float c) {
    c = fmaf(__uint_as_float(a.x), __uint_as_float(b.x), c);
    c = fmaf(__uint_as_float(a.y), __uint_as_float(b.y), c);
    c = fmaf(__uint_as_float(a.z), __uint_as_float(b.z), c);
    return fmaf(__uint_as_float(a.w), __uint_as_float(b.w), c);
}

// What a lane of a consumer warp has summed of a 16 x 8 tile: in the layout of
// the mma's accumulator, rows g and g + 8, columns 2 q and 2 q + 1 (g = lane / 4,
// q = lane % 4).
template <typename T> struct Acc;

template <> struct Acc<__nv_bfloat16> {
    float c[4];
    __device__ __forceinline__ void clear() { c[0] = c[1] = c[2] = c[3] = 0.f; }
    // one step: slot holds this lane's 16 bytes of rows g and g + 8 and of the entry's row g
    __device__ __forceinline__ void step(const char *slot, int, int lane) {
        const uint4 lo = *reinterpret_cast<const uint4 *>(slot + lane * 16);
        const uint4 hi = *reinterpret_cast<const uint4 *>(slot + 512 + lane * 16);
        // columns past the entry's rows hold anything; they are not stored
        const uint4 bb = *reinterpret_cast<const uint4 *>(slot + 1024 + lane * 16);
        mma_bf16(c, lo.x, hi.x, lo.y, hi.y, bb.x, bb.y);
        mma_bf16(c, lo.z, hi.z, lo.w, hi.w, bb.z, bb.w);
    }
    __device__ __forceinline__ void get(float (&v)[4], int) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = c[i];
    }
};

template <> struct Acc<float> {
    float lo[FW_N], hi[FW_N];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < FW_N; ++n) lo[n] = hi[n] = 0.f;
    }
    __device__ __forceinline__ void step(const char *slot, int cnt, int lane) {
        const uint4 al = *reinterpret_cast<const uint4 *>(slot + lane * 16);
        const uint4 ah = *reinterpret_cast<const uint4 *>(slot + 512 + lane * 16);
#pragma unroll
        for (int n = 0; n < FW_N; ++n) {
            if (n >= cnt) break;
            const uint4 bb = *reinterpret_cast<const uint4 *>(slot + 1024 + n * 64 + (lane & 3) * 16);
            lo[n] = dot16<float>(al, bb, lo[n]);
            hi[n] = dot16<float>(ah, bb, hi[n]);
        }
    }
    // the four lanes of a row hold every fourth 16 bytes of it
    __device__ __forceinline__ void get(float (&v)[4], int lane) {
        const int q = lane & 3;
#pragma unroll
        for (int n = 0; n < FW_N; ++n) {
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                lo[n] += __shfl_xor_sync(0xffffffffu, lo[n], o);
                hi[n] += __shfl_xor_sync(0xffffffffu, hi[n], o);
            }
        }
        v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
        for (int n = 0; n < FW_N; ++n)
            if ((n >> 1) == q) {
                v[n & 1] = lo[n];
                v[2 + (n & 1)] = hi[n];
            }
    }
};

// Shared memory, in bytes: the ring, the warps' sums, out's sums, the tables of
// the T k (token, slot) pairs.
__host__ __device__ inline int few_ring_bytes(int depth) { return FW_WARPS * depth * FW_SLOT; }
constexpr int kFewRed = 2 * FW_WARPS * 32 * 16;
__host__ __device__ inline int few_out_bytes(int T) { return FW_WARPS * FW_M * T * 4; }
__host__ __device__ inline int few_table_bytes(int slots) { return slots * 16 + 16; }

// Key of expert e for every token, by the CTA's warps.
template <typename T>
__device__ __forceinline__ void few_route(const FewParams &p, float *s_part, int warp, int lane) {
    constexpr int EPV = 16 / (int)sizeof(T);
    const int G = gridDim.x, vecs = p.D / EPV;
    const int mine = p.E > (int)blockIdx.x ? (p.E - (int)blockIdx.x + G - 1) / G : 0;
    if (mine == 0) return;
    int side = 1;  // experts side by side, 8 / side warps each
    while (side < mine && side < FW_WARPS) side <<= 1;
    const int wpe = FW_WARPS / side, sub = warp % wpe;
    for (int i0 = 0; i0 < mine; i0 += side) {
        const int i = i0 + warp / wpe;
        const int e = blockIdx.x + i * G;
        for (int t0 = 0; t0 < p.T; t0 += FW_N) {
            float acc[FW_N];
#pragma unroll
            for (int n = 0; n < FW_N; ++n) acc[n] = 0.f;
            if (i < mine) {
                const uint4 *w = static_cast<const uint4 *>(p.wg) + (size_t)e * vecs;
                const uint4 *x = static_cast<const uint4 *>(p.x) + (size_t)t0 * vecs;
#pragma unroll 4
                for (int v = sub * 32 + lane; v < vecs; v += wpe * 32) {
                    const uint4 wv = w[v];
#pragma unroll
                    for (int n = 0; n < FW_N; ++n)
                        if (t0 + n < p.T) acc[n] = dot16<T>(wv, x[(size_t)n * vecs + v], acc[n]);
                }
            }
#pragma unroll
            for (int n = 0; n < FW_N; ++n) {
                if (t0 + n >= p.T) break;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[n] += __shfl_xor_sync(0xffffffffu, acc[n], o);
                if (lane == 0) s_part[warp * FW_N + n] = acc[n];
            }
            __syncthreads();
            const int at = warp * 32 + lane;  // (expert side by side, token)
            if (at < side * FW_N) {
                const int j = at / FW_N, n = at % FW_N;
                if (i0 + j < mine && t0 + n < p.T) {
                    const int ej = blockIdx.x + (i0 + j) * G;
                    float key = 0.f;
                    for (int u = 0; u < wpe; ++u) key += s_part[(j * wpe + u) * FW_N + n];
                    if (p.bias) key += p.bias[ej];
                    p.logits[(size_t)(t0 + n) * p.E + ej] = key;
                }
            }
            __syncthreads();
        }
    }
}

// DEPTH: steps of a warp in flight.
template <typename T, int DEPTH>
__global__ void __launch_bounds__(FW_THREADS, 1)
few_layer_kernel(const FewParams p) {
    extern __shared__ __align__(128) char smem[];
    __shared__ volatile int s_abort;
    __shared__ int s_local, s_entries, s_last[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = gridDim.x;
    const int slots = p.T * p.k;
    char *ring = smem + warp * DEPTH * FW_SLOT;  // this warp's
    float4 *s_red = reinterpret_cast<float4 *>(smem + few_ring_bytes(DEPTH));  // [2][warps][32]
    float *s_out = reinterpret_cast<float *>(s_red + 2 * FW_WARPS * 32);       // [warps][T][16]
    float *s_w = s_out + FW_WARPS * FW_M * p.T;                                // [slots]
    int *s_idx = reinterpret_cast<int *>(s_w + slots);                         // [slots]
    int *s_sorted = s_idx + slots;  // [slots]: slot of the n-th pair in order of (expert, slot)
    uint32_t *s_entry = reinterpret_cast<uint32_t *>(s_sorted + slots);  // [entries + 1]: expert << 16 | first pair
    constexpr int EB = (int)sizeof(T);

    griddep_wait();
    if (tid == 0) s_abort = 0;
    __syncthreads();

    // ---- route ----
    if (p.phases & FEW_ROUTE) {
        few_route<T>(p, reinterpret_cast<float *>(s_red), warp, lane);
        __syncthreads();
        if (p.phases != FEW_ALL) return;
        if (tid == 0) {
            fence_acq_rel_gpu();
            red_release_gpu_add(&p.bars[0], 1);
            wait_count_bounded(&p.bars[0], G, &s_abort);
        }
        __syncthreads();
    }
    bool dead = s_abort;  // the same for every thread: set before the barrier only
    // ---- top-k and the entries, every CTA for itself ----
    if (!dead) {
        for (int t = warp; t < p.T; t += FW_WARPS)
            warp_topk_weights<1024>(p.logits + (size_t)t * p.E, p.E, p.k, p.score, p.renorm,
                                    p.n_group, p.topk_group, t, s_idx, s_w,
                                    blockIdx.x == 0 ? p.status : nullptr, lane);
    }
    __syncthreads();
    if (!dead) {
        for (int i = tid; i < slots; i += FW_THREADS) {
            const int e = s_idx[i] - p.e_first;
            int place = 0, same = 0;
            for (int j = 0; j < slots; ++j) {
                const int ej = s_idx[j] - p.e_first;
                if (ej < 0 || ej >= p.E_local) continue;
                if (ej < e || (ej == e && j < i)) ++place;
                if (ej == e && j < i) ++same;
            }
            if (e >= 0 && e < p.E_local) {
                s_sorted[place] = i;
                // the pair's expert, and whether it begins an entry; read by warp 0 below
                s_entry[place] = (uint32_t)e << 16 | (same % FW_N == 0 ? 1u : 0u);
            }
        }
    }
    if (tid == 0) s_local = 0;
    __syncthreads();
    if (warp == 0 && !dead) {
        int local = 0;
        for (int i = lane; i < slots; i += 32) {
            const int e = s_idx[i] - p.e_first;
            local += e >= 0 && e < p.E_local;
        }
        local = __reduce_add_sync(0xffffffffu, local);
        int n = 0;  // entries so far; never ahead of the pairs read
        for (int b = 0; b < local; b += 32) {
            const uint32_t v = b + lane < local ? s_entry[b + lane] : 0u;
            const bool first = v & 1u;
            const uint32_t m = __ballot_sync(0xffffffffu, first);
            if (first) s_entry[n + __popc(m & lanemask_lt())] = (v & 0xffff0000u) | (uint32_t)(b + lane);
            n += __popc(m);
            __syncwarp();
        }
        if (lane == 0) {
            s_entry[n] = (uint32_t)local;
            s_local = local;
            s_entries = n;
        }
    }
    __syncthreads();

    const int U = s_local ? s_entries : 0;
    auto first_of = [&](int u) { return (int)(s_entry[u] & 0xffffu); };
    // A warp's copies: its next step's row pieces (this lane's of rows g, g + 8
    // and of the entry's row g) and how far the row goes on behind them.
    const int g = lane >> 2, col = warp * FW_STEP + (lane & 3) * 16;
    const char *lo = nullptr, *hi = nullptr, *row = nullptr;
    bool has_lo = false, has_hi = false, has_row = false;  // this lane has such a row
    int left = 0;     // bytes of the row from this lane's piece on; <= 0: past its end
    int in_slot = 0;  // ring slot of the next copies, of the next step
    int out_slot = 0;
    const char *any = static_cast<const char *>(p.x);  // a valid address for copies of nothing
    auto copy_weights = [&](int slot) {
        char *d = ring + slot * FW_SLOT + lane * 16;
        const bool in_lo = left > 0 && has_lo, in_hi = left > 0 && has_hi;
        copy16(d, in_lo ? lo : any, in_lo);
        copy16(d + 512, in_hi ? hi : any, in_hi);
    };
    auto copy_row = [&](int slot) {
        if (has_row) copy16(ring + slot * FW_SLOT + 1024 + lane * 16, left > 0 ? row : any, left > 0);
    };
    auto advance = [&]() {
        lo += FW_CHUNK;
        hi += FW_CHUNK;
        row += FW_CHUNK;
        left -= FW_CHUNK;
    };
    auto bump = [&](int &slot) { slot = slot + 1 == DEPTH ? 0 : slot + 1; };
    Acc<T> acc;
    int turn = 0;

    // ---- GEMM1: tiles of 8 hidden units of one entry ----
    if ((p.phases & FEW_GEMM1) && !dead) {
        const int nt = p.H / 8, row_bytes = p.D * EB, nc = (row_bytes + FW_CHUNK - 1) / FW_CHUNK;
        const int tiles = U * nt;
        int li = blockIdx.x, lc = nc;  // tile being copied, its chunks copied so far
        bool begun = false;
        auto copy_next = [&]() {
            if (lc == nc) {
                if (begun) li += G;
                begun = true;
                lc = 0;
                if (li < tiles) {
                    const int u = li / nt, j = li - u * nt;
                    const int e = s_entry[u] >> 16, f = first_of(u), cnt = first_of(u + 1) - f;
                    const size_t at = ((size_t)e * p.H + (size_t)j * 8 + g) * row_bytes + col;
                    lo = static_cast<const char *>(p.w1) + at;
                    hi = static_cast<const char *>(p.w3) + at;
                    has_row = g < cnt;
                    row = static_cast<const char *>(p.x) +
                          (has_row ? (size_t)(s_sorted[f + g] / p.k) * row_bytes : 0) + col;
                    left = row_bytes - col;
                    has_lo = has_hi = true;
                }
            }
            if (li < tiles) {
                copy_weights(in_slot);
                copy_row(in_slot);
                bump(in_slot);
                advance();
                ++lc;
            } else {
                lc = 0;  // stay past the end
                begun = false;
            }
            copy_commit();
        };
        for (int i = 0; i < DEPTH - 1; ++i) copy_next();
        for (int i = blockIdx.x; i < tiles; i += G) {
            const int u = i / nt, j = i - u * nt;
            const int f = first_of(u), cnt = first_of(u + 1) - f;
            acc.clear();
            for (int c = 0; c < nc; ++c) {
                copy_wait<DEPTH - 2>();
                __syncwarp();
                acc.step(ring + out_slot * FW_SLOT, cnt, lane);
                bump(out_slot);
                copy_next();  // into the slot read a step ago
            }
            float v[4];
            acc.get(v, lane);
            float4 *red = s_red + turn * FW_WARPS * 32;
            turn ^= 1;  // the other buffer's readers are behind the barrier before this one
            red[warp * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
            __syncthreads();
            if (tid < 64) {
                // thread (lane, half): gate and up of unit lane / 4 for row 2 (lane % 4) + half
                const int half = tid >> 5, n = 2 * (lane & 3) + half;
                float gate = 0.f, up = 0.f;
#pragma unroll
                for (int w = 0; w < FW_WARPS; ++w) {
                    const float *r = reinterpret_cast<const float *>(&red[w * 32 + lane]);
                    gate += r[half];
                    up += r[2 + half];
                }
                if (n < cnt)
                    static_cast<T *>(p.h)[(size_t)(f + n) * p.H + j * 8 + g] =
                        Elem<T>::round(gate / (1.f + expf(-gate)) * up);
            }
        }
        copy_wait<0>();
        __syncwarp();
        if (p.phases == FEW_ALL) {
            __syncthreads();
            if (tid == 0) {
                fence_acq_rel_gpu();
                red_release_gpu_add(&p.bars[1], 1);
            }
            griddep_launch_dependents();
        }
    }

    // ---- GEMM2: this CTA's part of the line of (tile, entry, chunk) ----
    const int nt2 = (p.D + FW_M - 1) / FW_M;
    if ((p.phases & FEW_GEMM2) && !dead && U == 0) {  // no token has an expert here
        T *out = static_cast<T *>(p.out);
        for (long long i = (long long)blockIdx.x * FW_THREADS + tid; i < (long long)p.T * p.D;
             i += (long long)G * FW_THREADS)
            out[i] = Elem<T>::round(0.f);
    } else if ((p.phases & FEW_GEMM2) && !dead) {
        const int row_bytes = p.H * EB, nc = (row_bytes + FW_CHUNK - 1) / FW_CHUNK;
        const long long per_tile = (long long)U * nc, line = per_tile * nt2;
        // CTAs that take a part: no more than there are chunks, so that none is empty
        const int G2 = (int)min((long long)G, line);
        const bool part_of = (int)blockIdx.x < G2;
        const long long first = part_of ? line * blockIdx.x / G2 : 0;
        const int total = part_of ? (int)(line * (blockIdx.x + 1) / G2 - first) : 0;
        const int dt0 = (int)(first / per_tile);
        const int u0 = (int)((first - dt0 * per_tile) / nc), c0 = (int)(first - dt0 * per_tile) - u0 * nc;
        // copy cursor
        int ln = 0, ldt = dt0, lu = u0, lc = c0;
        auto set_weights = [&](int dt, int u, int c) {
            const int e = s_entry[u] >> 16, d = dt * FW_M + g;
            const size_t at = ((size_t)e * p.D + d) * row_bytes + (size_t)c * FW_CHUNK + col;
            has_lo = d < p.D;  // D is a multiple of 8: rows g all are, rows g + 8 may not be
            has_hi = d + 8 < p.D;
            lo = static_cast<const char *>(p.w2) + (has_lo ? at : 0);
            hi = static_cast<const char *>(p.w2) + (has_hi ? at + (size_t)8 * row_bytes : 0);
            left = row_bytes - c * FW_CHUNK - col;
        };
        auto set_row = [&](int u, int c) {
            const int f = first_of(u), cnt = first_of(u + 1) - f;
            has_row = g < cnt;
            row = static_cast<const char *>(p.h) + (size_t)(f + (has_row ? g : 0)) * row_bytes +
                  (size_t)c * FW_CHUNK + col;
            left = row_bytes - c * FW_CHUNK - col;
        };
        auto step_on = [&](int &dt, int &u, int &c) {  // true: another entry or tile begins
            if (++c < nc) return false;
            c = 0;
            if (++u == U) {
                u = 0;
                ++dt;
            }
            return true;
        };
        // the weights of the first steps go out before the barrier, the rows (h) behind it
        const int ahead = min(DEPTH - 1, total);
        int dt = dt0, u = u0, c = c0;
        for (int i = 0; i < ahead; ++i) {
            if (i == 0 || c == 0) set_weights(dt, u, c);
            copy_weights((in_slot + i) % DEPTH);
            advance();
            step_on(dt, u, c);
        }
        if (p.phases == FEW_ALL) {
            if (tid == 0) wait_count_bounded(&p.bars[1], G, &s_abort);
            __syncthreads();
            dead = s_abort;
        }
        if (!dead) {
            for (int i = 0; i < DEPTH - 1; ++i) {
                if (i < ahead) {
                    if (i == 0 || lc == 0) set_row(lu, lc);
                    copy_row(in_slot);
                    bump(in_slot);
                    advance();
                    step_on(ldt, lu, lc);
                    ++ln;
                }
                copy_commit();
            }
            if (ln < total) {
                set_weights(ldt, lu, lc);
                set_row(lu, lc);
            }
            auto copy_next = [&]() {
                if (ln < total) {
                    copy_weights(in_slot);
                    copy_row(in_slot);
                    bump(in_slot);
                    advance();
                    ++ln;
                    if (step_on(ldt, lu, lc) && ln < total) {
                        set_weights(ldt, lu, lc);
                        set_row(lu, lc);
                    }
                }
                copy_commit();
            };
            for (int i = lane; i < FW_M * p.T; i += 32) s_out[warp * FW_M * p.T + i] = 0.f;
            __syncwarp();
            T *out = static_cast<T *>(p.out);
            dt = dt0, u = u0, c = c0;
            int cut[2] = {-1, -1};  // tiles that others share: the first, the last
            for (int n = 0; n < total;) {
                const bool from_start = u == 0 && c == 0;
                bool to_end = false;
                while (n < total && !to_end) {  // this CTA's part of one entry
                    const int f = first_of(u), cnt = first_of(u + 1) - f;
                    acc.clear();
                    bool more = true;
                    while (more && n < total) {
                        copy_wait<DEPTH - 2>();
                        __syncwarp();
                        acc.step(ring + out_slot * FW_SLOT, cnt, lane);
                        bump(out_slot);
                        copy_next();
                        ++n;
                        more = ++c < nc;
                    }
                    if (!more) {
                        c = 0;
                        to_end = ++u == U;
                    }
                    float v[4];
                    acc.get(v, lane);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int m = 2 * (lane & 3) + half;
                        if (m >= cnt) continue;
                        const int slot = s_sorted[f + m];
                        float *o = s_out + (warp * p.T + slot / p.k) * FW_M;
                        o[g] = fmaf(s_w[slot], v[half], o[g]);
                        o[g + 8] = fmaf(s_w[slot], v[2 + half], o[g + 8]);
                    }
                    __syncwarp();
                }
                // the warps' sums; a tile that others share goes through memory
                const bool whole = from_start && to_end;
                float *part = p.part + ((size_t)blockIdx.x * 2 + (dt == dt0 ? 0 : 1)) * p.T * FW_M;
                if (!whole) cut[dt == dt0 ? 0 : 1] = dt;
                __syncthreads();
                for (int o = tid; o < FW_M * p.T; o += FW_THREADS) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < FW_WARPS; ++w) {
                        sum += s_out[w * FW_M * p.T + o];
                        s_out[w * FW_M * p.T + o] = 0.f;
                    }
                    const int d = dt * FW_M + o % FW_M;
                    if (!whole)
                        part[o] = sum;
                    else if (d < p.D)
                        out[(size_t)(o / FW_M) * p.D + d] = Elem<T>::round(sum);
                }
                __syncthreads();
                u = 0;
                ++dt;
            }
            // shared tiles: the CTA that comes last adds the parts, in order
            int ca[2], cb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (cut[i] < 0) continue;
                const long long a0 = cut[i] * per_tile, a1 = a0 + per_tile;
                ca[i] = cb[i] = (int)blockIdx.x;
                while (ca[i] > 0 && line * ca[i] / G2 > a0) --ca[i];
                while (line * (cb[i] + 1) / G2 < a1) ++cb[i];
            }
            if (tid < 2) {
                const int mine = tid == 0 ? cut[0] : cut[1];
                if (mine >= 0) {
                    fence_acq_rel_gpu();
                    const int before = atomicAdd(&p.tile_count[mine], 1);
                    fence_acq_rel_gpu();
                    s_last[tid] = before == (tid == 0 ? cb[0] - ca[0] : cb[1] - ca[1]);
                    if (s_last[tid]) p.tile_count[mine] = 0;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (cut[i] < 0 || !s_last[i]) continue;
                for (int o = tid; o < FW_M * p.T; o += FW_THREADS) {
                    float sum = 0.f;
                    for (int b = ca[i]; b <= cb[i]; ++b) {
                        const int theirs = (int)(line * b / G2 / per_tile);
                        sum += __ldcg(p.part + ((size_t)b * 2 + (cut[i] == theirs ? 0 : 1)) * p.T * FW_M + o);
                    }
                    const int d = cut[i] * FW_M + o % FW_M;
                    if (d < p.D) out[(size_t)(o / FW_M) * p.D + d] = Elem<T>::round(sum);
                }
            }
        }
        copy_wait<0>();
    }
    __syncthreads();
    if (tid == 0) {
        const bool aborted = s_abort;
        if (aborted) raise_flag(p.status, FLAG_TIMEOUT);
        if (p.phases == FEW_ALL) {
            // the last CTA to leave puts the counters back
            fence_acq_rel_gpu();
            if (atomicAdd(&p.bars[2], 1) == G - 1) {
                fence_acq_rel_gpu();
                if (atomicOr(p.status, 0) & FLAG_TIMEOUT)  // some parts never came
                    for (int i = 0; i < nt2; ++i) p.tile_count[i] = 0;
                p.bars[0] = p.bars[1] = p.bars[2] = 0;
            }
        }
    }
}

}  // namespace

int64_t few_scratch_ints(int D) { return 64 + (D + FW_M - 1) / FW_M; }
int64_t few_part_floats(int T) { return (int64_t)kFewMaxCtas * 2 * T * FW_M; }

cudaError_t launch_few_layer(const FewLayer &f, cudaStream_t stream) {
    FewParams p = {};
    p.x = f.x;
    p.wg = f.wg;
    p.bias = f.bias;
    p.w1 = f.w1;
    p.w3 = f.w3;
    p.w2 = f.w2;
    p.out = f.out;
    p.h = f.h;
    p.logits = f.logits;
    p.part = f.part;
    p.bars = f.counters;
    p.tile_count = f.counters + 64;
    p.status = f.status;
    p.T = f.T;
    p.D = f.D;
    p.H = f.H_local;
    p.E = f.E;
    p.k = f.k;
    p.e_first = f.e_first;
    p.E_local = f.E_local;
    p.score = f.score;
    p.renorm = f.renorm;
    p.n_group = f.n_group;
    p.topk_group = f.topk_group;
    // 8 steps of every warp in flight (128 KB of weights per SM), 6 where many
    // tokens' sums take the shared memory
    const bool deep = f.T <= 8;
    const size_t smem = (size_t)few_ring_bytes(deep ? 8 : 6) + kFewRed + few_out_bytes(f.T) +
                        few_table_bytes(f.T * f.k);
    auto fn = f.is_bf16 ? (deep ? few_layer_kernel<__nv_bfloat16, 8> : few_layer_kernel<__nv_bfloat16, 6>)
                        : (deep ? few_layer_kernel<float, 8> : few_layer_kernel<float, 6>);
    cudaError_t err = ensure_smem((const void *)fn, smem);
    if (err != cudaSuccess) return err;
    const int ctas = std::min(sm_count(), kFewMaxCtas);
    if (ctas <= 0) return cudaErrorInvalidDevice;
    // A device (or a partition of one) that cannot hold the whole grid at once
    // refuses the cooperative launch, and under a profiler such launches have
    // failed: the three stages are then launched one by one.  MOE_FEW_LAUNCHES=3
    // asks for that.
    const char *sel = getenv("MOE_FEW_LAUNCHES");
    if (!(sel && strcmp(sel, "3") == 0) && !profiler_attached()) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(FW_THREADS);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeCooperative;
        attr[0].val.cooperative = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        p.phases = FEW_ALL;
        err = cudaLaunchKernelEx(&cfg, fn, p);
        if (err == cudaSuccess) count_launch();
        if (err != cudaErrorCooperativeLaunchTooLarge && err != cudaErrorNotSupported) return err;
        cudaGetLastError();
    }
    for (const int phases : {FEW_ROUTE, FEW_GEMM1, FEW_GEMM2}) {
        p.phases = phases;
        err = launch_pdl(fn, dim3(ctas), dim3(FW_THREADS), smem, stream, p);
        if (err != cudaSuccess) return err;
        count_launch();
    }
    return cudaSuccess;
}

}  // namespace moe
