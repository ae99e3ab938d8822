// The whole layer for a few tokens, in one kernel.
//
//   key = x Wg^T + b, top-k and weights w;  h_j = SiLU(w1_e x) * (w3_e x);
//   out[t] = sum_j w_j (w2_e h_j),  e = the token's j-th expert.
//
// With T <= 32 tokens a weight of a chosen expert is mostly used for a handful of
// rows, so the layer is bound by streaming the chosen experts' weights from HBM
// (3 D H values each), and by the latency of whatever stands before that stream.
// Launched as five steps, the steps' launches and tails cost about as much as
// the stream itself; here one CTA per SM runs all of them, with two barriers
// across the grid (cooperative launch):
//
//   route    expert rows of Wg over the CTAs, one dot product per token
//   -- barrier -- every CTA selects all tokens' experts for itself and sorts the
//            (token, slot) pairs by expert; at most 4 pairs of an expert (fp32:
//            8) form an ENTRY, one pass over that expert's weights
//   GEMM1    tiles of 8 gate and 8 up rows of one entry over the CTAs -> h
//   -- barrier --
//   GEMM2    tiles of 16 rows of out; all (tile, entry, chunk of H) triples in
//            one line, cut into equal parts over the CTAs, so that the stream
//            ends everywhere at once.  A tile cut by that gets its parts' fp32
//            sums through memory, added by the CTA that comes last, in order.
//
// The 16 weight rows of a tile are the M side of mma.sync m16n8k16 and the
// entry's rows the N = 8 side: at 8 rows per weight the tensor pipe idles either
// way, and register accumulators need no TMEM round trip.  The CTA's 8 warps
// split k: of every 2 KB of a row a warp takes 256 bytes (short rows: see below),
// copied with cp.async into a ring of its own and read back as 16-byte pieces (the
// sum over k does not care which k meet in one instruction, as long as both
// operands agree), so the stream needs no barrier but the sum over the warps at a
// tile's end, and the copies of the next tiles run through it.  (Bulk copies by a
// producer warp: each costs 55 ns to issue whatever its size, so 16 row pieces of
// 1 KB per stage reached 39% of the copy rate, of 4 KB 97% in long rows.  A dry
// pass of the loops under the first barrier, to have their instructions fetched:
// one token 32.9 us against 32.0.)
// fp32 layers use the same tiles with fused multiply-adds.
//
// Measured (GB300, bf16): 16 tokens over 256 experts of 7168 x 2048, 9.0 GB of
// weights, 1.24-1.29 ms (7.0-7.3 TB/s, the copy rate is 6.8); 8 tokens of the
// fine-grained layer, 0.60 GB, 108-110 us (5.5-5.6 TB/s); one token of it, 104 MB,
// 33.0 us, of which the stream's floor is 15.3.  The rest is latency: keys 2 us,
// barrier 1.3, top-k 2.4, entries 1.2, 4-6 until the first weights are there
// (address translation and DRAM), the second barrier 2, and all of it run once, so
// that its instructions come from L2.  (The layer's own calls take 64 us.)
// An expert with more pairs than an entry holds is streamed again, and GEMM1 runs
// an entry's tiles before the next entry, so from HBM where its weights are large:
// 8 experts of 4096 x 14336, two a token, take 416 us for 8 tokens, 505 for 12 and
// 810 for 32, where the layer's own calls take 430, 468 and 471.
//
// Rounding: keys, weights, both products' sums and the sum over experts are
// fp32; out is rounded once.  h of a bf16 layer goes to the second product as the
// sum of two bf16 (16 significant bits): four pairs' second parts take the columns
// that an entry of four leaves free, and out is off by its own rounding alone (h
// in one bf16: 0.0023-0.0027 of the RMS against 64 bits, in two 0.0017).  That
// holds an entry to four pairs, in the first product too: 32 tokens on 13 of 20
// experts of 1048 x 424 take 43.5 us, with entries of eight and h in one bf16 they
// took 33.4.  Where w2 is infinite the first part alone counts.  Every sum has a
// fixed order for a given grid, so results do not change from run to run.
#include <algorithm>

#include <stdlib.h>
#include <string.h>

#include "common.cuh"
#include "launch.h"
#include "topk.cuh"

namespace moe {
namespace {

constexpr int FW_WARPS = 8;
constexpr int FW_THREADS = 32 * FW_WARPS;
constexpr int FW_STEP = 256;                   // bytes of a row that a warp takes at once
constexpr int FW_M = 16;                       // weight rows per tile
constexpr int FW_N = 8;                        // the most rows of an entry (bf16: half as many)
constexpr int FW_SMEM = 226 * 1024;            // of the 227 KB a CTA may have
constexpr int FW_JOIN = 8192;                  // bytes of a row as long as joining a shared tile's parts takes

enum { FEW_ROUTE = 1, FEW_GEMM1 = 2, FEW_GEMM2 = 4, FEW_ALL = 7 };

struct FewParams {
    const void *x, *wg, *w1, *w3, *w2;
    const float *bias;
    void *out, *h;     // h: [T k][H] by the pair's place in the sorted order (bf16: [2][T k][H])
    float *logits;     // [T][E]
    float *part;       // [gridDim.x][2][T][16]
    int *bars;         // [0], [1] the grid barriers, [2] CTAs done; zero between calls
    // Parts in of the shared tile that CTA b holds the first part of: half word b
    // (one tile at most goes on behind b's part); zero between calls.
    unsigned *tile_count;
    int *status;
    int T, D, H, E, k, e_first, E_local, score, renorm, n_group, topk_group;
    int rows;  // pairs of an entry, at most
    int phases;
};

template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float round(float v) { return v; }
    static __device__ __forceinline__ void put(float v, float *h, float *) { *h = v; }
};
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
    // v as the sum of two bf16; what is not finite has no second part
    static __device__ __forceinline__ void put(float v, __nv_bfloat16 *h, __nv_bfloat16 *low) {
        *h = round(v);
        const float first = __bfloat162float(*h);
        *low = round(fabsf(first) < INFINITY ? v - first : 0.f);
    }
};

// 16 bytes global -> shared, past L1; zeros when !in (nothing is read then,
// wherever src points).
__device__ __forceinline__ void copy16(uint32_t dst, const char *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
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

// A step in the ring: two halves of 128 bytes of a row; in each, 16 weight rows,
// then the entry's rows, 128 bytes of each in 16-byte pieces.  Odd rows have
// their 64 bytes exchanged: lanes 8 i .. 8 i + 7 read 64 bytes of two rows at
// once, which so lie in different banks.
constexpr int FW_LINE = 128;
__device__ __forceinline__ int piece_at(int row, int piece) {
    return row * FW_LINE + (piece ^ ((row & 1) << 2)) * 16;
}

// What a lane of a warp has summed of a 16 x 8 tile: in the layout of the mma's
// accumulator, rows g and g + 8, columns 2 q and 2 q + 1 (g = lane / 4, q = lane % 4).
template <typename T> struct Acc;

template <> struct Acc<__nv_bfloat16> {
    float c[2][4];  // two chains of products
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[0][i] = c[1][i] = 0.f;
    }
    // lows: 0, or where the second parts of the entry's rows (columns 4 ..) begin
    __device__ __forceinline__ void step(const char *slot, int half_bytes, int cnt, int lows, int lane) {
        const int g = lane >> 2, row = FW_M + (lows && g >= 4 ? lows + g - 4 : g);
        const bool there = (lows ? g & 3 : g) < cnt;
        const char *at = slot + piece_at(g, lane & 3), *bt = slot + piece_at(row, lane & 3);
        const int other = piece_at(g, (lane & 3) + 4) - piece_at(g, lane & 3);
        const int other_b = piece_at(row, (lane & 3) + 4) - piece_at(row, lane & 3);
#pragma unroll
        for (int half = 0; half < 2; ++half, at += half_bytes, bt += half_bytes)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const char *a = at + k * other;
                const uint4 lo = *reinterpret_cast<const uint4 *>(a);
                const uint4 hi = *reinterpret_cast<const uint4 *>(a + 8 * FW_LINE);
                uint4 bb = make_uint4(0, 0, 0, 0);
                if (there) bb = *reinterpret_cast<const uint4 *>(bt + k * other_b);
                mma_bf16(c[0], lo.x, hi.x, lo.y, hi.y, bb.x, bb.y);
                mma_bf16(c[1], lo.z, hi.z, lo.w, hi.w, bb.z, bb.w);
            }
    }
    __device__ __forceinline__ void get(float (&v)[4], int, int) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = c[0][i] + c[1][i];
    }
};

template <> struct Acc<float> {
    float lo[FW_N], hi[FW_N];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < FW_N; ++n) lo[n] = hi[n] = 0.f;
    }
    __device__ __forceinline__ void step(const char *slot, int half_bytes, int cnt, int, int lane) {
#pragma unroll
        for (int half = 0; half < 2; ++half, slot += half_bytes)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int piece = (lane & 3) + 4 * k, at = piece_at(lane >> 2, piece);
                const uint4 al = *reinterpret_cast<const uint4 *>(slot + at);
                const uint4 ah = *reinterpret_cast<const uint4 *>(slot + 8 * FW_LINE + at);
#pragma unroll
                for (int n = 0; n < FW_N; ++n) {
                    if (n >= cnt) break;
                    const uint4 bb =
                        *reinterpret_cast<const uint4 *>(slot + FW_M * FW_LINE + piece_at(n, piece));
                    lo[n] = dot16<float>(al, bb, lo[n]);
                    hi[n] = dot16<float>(ah, bb, hi[n]);
                }
            }
    }
    // the four lanes of a row hold every fourth 16 bytes of it
    __device__ __forceinline__ void get(float (&v)[4], int cnt, int lane) {
        const int q = lane & 3;
#pragma unroll
        for (int n = 0; n < FW_N; ++n) {
            if (n >= cnt) break;
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

// Shared memory, in bytes: the ring, the warps' sums (GEMM1's two buffers of a
// tile, then GEMM2's of out), the tables of the T k (token, slot) pairs.
template <typename T> constexpr bool kFewSplit = sizeof(T) == 2;  // h in two parts
// Rows of an entry's pairs in the ring: fp32 `rows`, bf16 twice that (the parts of h).
__host__ __device__ inline int few_slot_bytes(int rows, bool split) {
    return (FW_M + (split ? 2 * rows : rows)) * FW_STEP;
}
__host__ __device__ inline int few_sum_bytes(int T) {
    return FW_WARPS * FW_M * 4 * (T > 16 ? T : 16);  // GEMM1: 2 x 32 lanes x 16 bytes a warp
}
__host__ __device__ inline int few_table_bytes(int slots) { return slots * 20 + 16; }

// Keys of tokens t0 .. t0 + NT - 1 for one expert: this warp's share (v0, v0 +
// stride, ...) of the dot products, summed over the lanes.
template <typename T, int NT>
__device__ __forceinline__ void few_dots(const FewParams &p, int e, int t0, int v0, int stride,
                                         int lane, float *to) {
    constexpr int EPV = 16 / (int)sizeof(T);
    const int vecs = p.D / EPV, n_here = min(NT, p.T - t0);
    const uint4 *w = static_cast<const uint4 *>(p.wg) + (size_t)e * vecs;
    const uint4 *x = static_cast<const uint4 *>(p.x) + (size_t)t0 * vecs;
    float acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = 0.f;
#pragma unroll 1
    for (int v = v0 + lane; v < vecs; v += stride) {
        const uint4 wv = w[v];
        uint4 xv[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) xv[n] = x[(size_t)min(n, n_here - 1) * vecs + v];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n] = dot16<T>(wv, xv[n], acc[n]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[n] += __shfl_xor_sync(0xffffffffu, acc[n], o);
        if (lane == 0) to[n] = acc[n];
    }
}

// The keys: (expert, group of 8 tokens) pairs over the CTAs, a CTA's own side by
// side over its warps.
template <typename T>
__device__ __forceinline__ void few_route(const FewParams &p, float *s_part, int tid) {
    const int warp = tid >> 5, lane = tid & 31, G = gridDim.x;
    const int groups = (p.T + FW_N - 1) / FW_N, units = p.E * groups;
    const int mine = units > (int)blockIdx.x ? (units - (int)blockIdx.x + G - 1) / G : 0;
    if (mine == 0) return;
    int side = 1;  // pairs side by side, FW_WARPS / side warps each
    while (side < mine && side < FW_WARPS) side <<= 1;
    const int wpe = FW_WARPS / side, sub = warp % wpe;
    for (int i0 = 0; i0 < mine; i0 += side) {
        const int i = i0 + warp / wpe, unit = blockIdx.x + i * G;
        if (i < mine) {
            const int e = unit / groups, t0 = (unit - e * groups) * FW_N;
            if (p.T == 1)
                few_dots<T, 1>(p, e, t0, sub * 32, wpe * 32, lane, s_part + warp * FW_N);
            else
                few_dots<T, FW_N>(p, e, t0, sub * 32, wpe * 32, lane, s_part + warp * FW_N);
        }
        __syncthreads();
        const int j = tid / FW_N, n = tid % FW_N;
        if (j < side && i0 + j < mine) {
            const int un = blockIdx.x + (i0 + j) * G, e = un / groups, t = (un - e * groups) * FW_N + n;
            if (t < p.T) {
                float key = 0.f;
                for (int u = 0; u < wpe; ++u) key += s_part[(j * wpe + u) * FW_N + n];
                if (p.bias) key += p.bias[e];
                p.logits[(size_t)t * p.E + e] = key;
            }
        }
        __syncthreads();
    }
}

// The T k (token, slot) pairs whose expert is here, an expert's pairs together
// and in order, cut into entries of at most p.rows.  s_sorted[n]: slot of the n-th
// pair, s_token[n]: its token, s_entry[u]: expert << 16 | first pair of entry u,
// with a last one that holds the number of pairs.  Returns the entries.
__device__ __forceinline__ int few_entries(const FewParams &p, int slots, const int *s_idx,
                                           int *s_sorted, int *s_token, uint32_t *s_entry,
                                           int *s_count, int tid) {
    const int lane = tid & 31;
    if (slots <= 32) {  // one warp, a lane per pair: experts in the order of their first pairs
        if (tid < 32) {
            const int e = lane < slots ? s_idx[lane] - p.e_first : -1;
            const bool here = e >= 0 && e < p.E_local;
            const uint32_t mates = __match_any_sync(0xffffffffu, here ? e : -1 - lane);
            const int lead = __ffs(mates) - 1, size = __popc(mates);
            int packed = here && lead == lane ? (size << 16) | ((size + p.rows - 1) / p.rows) : 0;
            const int own = packed;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {  // pairs and entries of the experts up to here
                const int v = __shfl_up_sync(0xffffffffu, packed, o);
                if (lane >= o) packed += v;
            }
            const int all = __shfl_sync(0xffffffffu, packed, 31);
            const int before = __shfl_sync(0xffffffffu, packed - own, lead);
            const int rank = __popc(mates & lanemask_lt()), place = (before >> 16) + rank;
            if (here) {
                s_sorted[place] = lane;
                s_token[place] = lane / p.k;
                if (rank % p.rows == 0)
                    s_entry[(before & 0xffff) + rank / p.rows] = (uint32_t)e << 16 | (uint32_t)place;
            }
            if (lane == 0) {
                s_entry[all & 0xffff] = (uint32_t)(all >> 16);
                *s_count = all & 0xffff;
            }
        }
        __syncthreads();
        return *s_count;
    }
    // a thread per pair: its place by counting
    for (int i = tid; i < slots; i += FW_THREADS) {
        const int e = s_idx[i] - p.e_first;
        const bool here = e >= 0 && e < p.E_local;
        int place = 0, same = 0;
        if (here)
#pragma unroll 4
            for (int j = 0; j < slots; ++j) {
                const int ej = s_idx[j] - p.e_first;
                const bool twin = ej == e && j < i;
                place += (ej >= 0 && ej < e) || twin;
                same += twin;
            }
        if (here) {
            s_sorted[place] = i;
            s_token[place] = i / p.k;
            // the pair's expert, and whether it begins an entry: for the first warp
            s_entry[place] = (uint32_t)e << 16 | (same % p.rows == 0 ? 1u : 0u);
        }
    }
    __syncthreads();
    if (tid < 32) {
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
            *s_count = n;
        }
    }
    __syncthreads();
    return *s_count;
}

// Log2 of the warps that share a row of `steps` steps: as many as it has steps for.
__device__ __forceinline__ int few_sharing(int steps) {
    return (steps > 1) + (steps > 2) + (steps > 4);
}
static_assert(FW_WARPS == 8, "few_sharing counts up to it");

// A line of `n` cut into `parts`: first of part b, and the part that holds x.
__device__ __forceinline__ int cut_first(int n, int parts, int b) {
    const int q = n / parts, r = n - q * parts;
    return q * b + min(b, r);
}
__device__ __forceinline__ int cut_holder(int n, int parts, int x) {
    const int q = n / parts, r = n - q * parts;
    return x < r * (q + 1) ? x / (q + 1) : r + (x - r * (q + 1)) / q;
}

// DEPTH: steps of a warp in flight.
template <typename T, int DEPTH>
__global__ void __launch_bounds__(FW_THREADS, 1)
few_layer_kernel(const FewParams p) {
    extern __shared__ __align__(128) char smem[];
    __shared__ volatile int s_abort;
    __shared__ int s_count, s_last[2];
    __shared__ uint64_t s_full[FW_WARPS][2], s_free[FW_WARPS][2];  // the groups' buffers of their sums
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = gridDim.x;
    const int slots = p.T * p.k;
    constexpr bool SPLIT = kFewSplit<T>;
    const int slot_bytes = few_slot_bytes(p.rows, SPLIT);
    char *ring = smem + warp * DEPTH * slot_bytes;  // this warp's
    const int half_bytes = slot_bytes / 2;
    float4 *s_red = reinterpret_cast<float4 *>(smem + FW_WARPS * DEPTH * slot_bytes);  // [2][warps][32]
    float *s_out = reinterpret_cast<float *>(s_red);                                   // [warps][T][16]
    float *s_w = s_out + few_sum_bytes(p.T) / 4;                                       // [slots]
    int *s_idx = reinterpret_cast<int *>(s_w + slots);                         // [slots]
    int *s_sorted = s_idx + slots;                                             // [slots]
    int *s_token = s_sorted + slots;                                           // [slots]
    uint32_t *s_entry = reinterpret_cast<uint32_t *>(s_token + slots);         // [slots + 1]
    constexpr int EB = (int)sizeof(T);

    griddep_wait();
    if (tid == 0) {
        s_abort = 0;
        const int ks = 1 << few_sharing((p.D * EB + FW_STEP - 1) / FW_STEP);
        for (int i = 0; i < 2 * FW_WARPS; ++i) {
            mbar_init(&s_full[i >> 1][i & 1], ks);
            mbar_init(&s_free[i >> 1][i & 1], 1);
        }
        fence_mbarrier_init();
    }
    __syncthreads();

    // ---- route ----
    if (p.phases & FEW_ROUTE) {
        few_route<T>(p, reinterpret_cast<float *>(s_red), tid);
        if (p.phases != FEW_ALL) return;
        if (tid == 0) {
            fence_acq_rel_gpu();
            red_release_gpu_add(&p.bars[0], 1);
            wait_count_bounded(&p.bars[0], G, &s_abort);
        }
        __syncthreads();
    }
    bool dead = s_abort;  // the same for every thread: set before the barrier only
    int U = 0;
    if (!dead) {  // top-k and the entries, every CTA for itself
        for (int t = warp; t < p.T; t += FW_WARPS)
            warp_topk_weights<1024>(p.logits + (size_t)t * p.E, p.E, p.k, p.score, p.renorm,
                                    p.n_group, p.topk_group, t, s_idx, s_w,
                                    blockIdx.x == 0 ? p.status : nullptr, lane);
        __syncthreads();
        U = few_entries(p, slots, s_idx, s_sorted, s_token, s_entry, &s_count, tid);
    }
    auto first_of = [&](int u) { return (int)(s_entry[u] & 0xffffu); };

    const int g = lane >> 2;
    const int r4 = lane >> 3, c16 = lane & 7;  // a copy takes 4 rows' 128 bytes
    const uint32_t to_piece = smem_u32(ring) + piece_at(r4, c16);
    // where a copy's second row goes: four on, or its first row's second part
    const uint32_t to_second = smem_u32(ring) + piece_at(FW_M + (SPLIT ? p.rows : 4) + r4, c16);
    const int nt2 = (p.D + FW_M - 1) / FW_M;
    int in_slot = 0, out_slot = 0;  // ring slot of the next copies, of the next step
    Acc<T> acc;

    // Both products run the same loops (the second finds them in the instruction
    // cache): a SEGMENT is a tile's rows against one entry, nc chunks long.  Where a
    // row is short, fewer than all warps share it and the groups of `ks` warps take
    // different segments (24 tokens, D = 160, H = 880: 39 us when
    // this was chosen, with all 8 on a row 47).
    //   GEMM1: tile = 8 hidden units; the U nt tiles over all CTAs' groups, tiles of
    //          an entry running fastest
    //   GEMM2: tile = 16 rows of out; this CTA's part of the line of chunks, entries
    //          running fastest, a tile's entries over the groups
#pragma unroll 1
    for (int second = 0; second < 2; ++second) {
        if (!(p.phases & (second ? FEW_GEMM2 : FEW_GEMM1)) || dead || U == 0) continue;
        const int row_bytes = (second ? p.H : p.D) * EB;
        const int steps = (row_bytes + FW_STEP - 1) / FW_STEP;
        const int lg = few_sharing(steps), ks = 1 << lg;
        const int groups = FW_WARPS >> lg, group = warp >> lg, chunk = ks * FW_STEP;
        const int nc = (steps + ks - 1) >> lg;
        const int nt = second ? nt2 : p.H / 8;
        int tile0, u0, c0 = 0;  // where this warp begins
        int G2 = G, per_tile = 0, line = 0, first = 0, end = 0;
        if (!second) {
            const int b = blockIdx.x * groups + group;
            u0 = b / nt;
            tile0 = b - u0 * nt;
        } else {
            per_tile = U * nc;
            line = per_tile * nt;
            // Cut anywhere, the parts are equal to a chunk, but tiles cut in two
            // cost a handshake at the end, as long as FW_JOIN bytes of a row take;
            // whole tiles where that is no longer.
            const bool whole_tiles =
                (long long)((nt + G - 1) / G * per_tile - line / G) * min(chunk, row_bytes) <= FW_JOIN;
            const int unit = whole_tiles ? per_tile : 1, units = line / unit;
            G2 = min(G, units);
            if ((int)blockIdx.x < G2) {
                first = cut_first(units, G2, blockIdx.x) * unit;
                end = cut_first(units, G2, blockIdx.x + 1) * unit;
            }
            tile0 = first / per_tile;
            const int r = first - tile0 * per_tile;
            u0 = r / nc;
            c0 = r - u0 * nc;
            if (whole_tiles) line = 0;  // no tile is shared
        }
        const int first_tile = tile0;
        const bool from_start = u0 == 0 && c0 == 0;
        if (second) {  // this group's first segment
            const int skip = (group - u0) & (groups - 1);
            if (skip) c0 = 0;
            u0 += skip;
            if (u0 >= U) {
                u0 = group;
                ++tile0;
                c0 = 0;
            }
            if (group >= U) tile0 = nt;  // none
        }
        const char *weights = static_cast<const char *>(second ? p.w2 : p.w1);
        const char *rows = static_cast<const char *>(second ? p.h : p.x);
        // from rows g of a tile to its rows g + 8: the up weights, or eight rows on
        const ptrdiff_t to_hi = second ? (ptrdiff_t)8 * row_bytes
                                       : static_cast<const char *>(p.w3) - weights;
        const ptrdiff_t to_4 = (ptrdiff_t)4 * row_bytes;
        const int tile_rows = second ? FW_M : 8, R = second ? p.D : p.H;
        const bool two = SPLIT && second;  // the rows are h's two parts
        auto next_segment = [&](int &tile, int &u) {
            if (second) {
                u += groups;
                if (u >= U) {
                    u = group;
                    ++tile;
                }
            } else {
                tile += G * groups;
                while (tile >= nt) {
                    tile -= nt;
                    ++u;
                }
            }
        };
        // chunks of the line in front of a segment's chunk c; GEMM1 has no line
        auto position = [&](int tile, int u, int c) { return (tile * U + u) * nc + c; };
        // The copies' cursor: a segment, its next chunk, and this lane's pieces
        // there of rows r4, r4 + 4 (and 8 on) and of the entry's rows r4, r4 + 4.
        // The warps take turns at a segment's first step: where a row is no whole
        // number of chunks, each gets as many steps as the others.
        int ltile = tile0, lu = u0, lc = c0, left = 0, turn0 = 0;
        bool fresh = true, has_hi = false;
        int lpos = position(ltile, lu, lc);
        bool ahead = second ? lpos < end : lu < U;
        bool has_row = false, has_second = false;
        const char *lo = nullptr, *hi = nullptr, *row = nullptr, *row_4 = nullptr;
        auto open = [&]() {
            const uint32_t entry = s_entry[lu];
            const int e = entry >> 16, f = entry & 0xffff, cnt = first_of(lu + 1) - f;
            const int first_row = ltile * tile_rows;
            const int col = lc * chunk + ((warp + turn0) & (ks - 1)) * FW_STEP + c16 * 16;
            lo = weights + (size_t)(e * R + first_row + r4) * row_bytes + col;
            hi = lo + to_hi;
            has_hi = !second || first_row + 8 < R;  // R is a multiple of 8
            has_row = r4 < cnt;
            has_second = two ? has_row : r4 + 4 < cnt;
            const int n = f + (has_row ? r4 : 0), n4 = two ? slots + n : f + (has_second ? r4 + 4 : 0);
            row = rows + (size_t)(second ? n : s_token[n]) * row_bytes + col;
            row_4 = rows + (size_t)(second ? n4 : s_token[n4]) * row_bytes + col;
            left = row_bytes - col;
            fresh = false;
        };
        auto copy_weights = [&](int slot) {
            const uint32_t d = to_piece + slot * slot_bytes;
            const bool in[2] = {left > 0, left > FW_LINE};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t dh = d + half * half_bytes;
                copy16(dh, lo + half * FW_LINE, in[half]);
                copy16(dh + 4 * FW_LINE, lo + to_4 + half * FW_LINE, in[half]);
                copy16(dh + 8 * FW_LINE, hi + half * FW_LINE, in[half] && has_hi);
                copy16(dh + 12 * FW_LINE, hi + to_4 + half * FW_LINE, in[half] && has_hi);
            }
        };
        auto copy_row = [&](int slot) {
            if (has_row) {
                const uint32_t d = to_piece + slot * slot_bytes + FW_M * FW_LINE;
                copy16(d, row, left > 0);
                copy16(d + half_bytes, row + FW_LINE, left > FW_LINE);
            }
            if (has_second) {
                const uint32_t d = to_second + slot * slot_bytes;
                copy16(d, row_4, left > 0);
                copy16(d + half_bytes, row_4 + FW_LINE, left > FW_LINE);
            }
        };
        auto bump = [&](int &slot) { slot = slot + 1 == DEPTH ? 0 : slot + 1; };
        auto copy_next = [&]() {
            if (ahead) {
                if (fresh) open();
                copy_weights(in_slot);
                copy_row(in_slot);
                bump(in_slot);
                lo += chunk;
                hi += chunk;
                row += chunk;
                row_4 += chunk;
                left -= chunk;
                if (++lc == nc) {
                    lc = 0;
                    turn0 += steps;
                    next_segment(ltile, lu);
                    if (groups > 1) lpos = position(ltile, lu, 0) - 1;
                    fresh = true;
                }
                ahead = second ? ++lpos < end : lu < U;
            }
            copy_commit();
        };
        auto step = [&](int cnt) {  // the oldest copies, and the next into the slot read a step ago
            copy_wait<DEPTH - 2>();
            __syncwarp();
            acc.step(ring + out_slot * slot_bytes, half_bytes, cnt, two ? p.rows : 0, lane);
            bump(out_slot);
            copy_next();
        };
        // h of every CTA.  (The first steps' weights do not need it, but copying
        // them ahead of the barrier measured the same: its loads then queue behind.)
        if (second && p.phases == FEW_ALL) {
            if (tid == 0) wait_count_bounded(&p.bars[1], G, &s_abort);
            __syncthreads();
            dead = s_abort;
            if (dead) break;
        }
#pragma unroll 1
        for (int i = 0; i < DEPTH - 1; ++i) copy_next();
        T *out = static_cast<T *>(p.out);
        int tile = tile0, u = u0, c = c0, turn = 0;
        int cut[2] = {-1, -1};  // tiles that others share: the first, the last
        if (second) {
            for (int i = lane; i < FW_M * p.T; i += 32) s_out[warp * FW_M * p.T + i] = 0.f;
            __syncwarp();
        }
        // GEMM1: all of the warp's segments.  GEMM2: tile by tile of the CTA's part,
        // with the CTA's sums at the end of each.
#pragma unroll 1
        for (int at = first_tile; second ? at * per_tile < end : at == first_tile; ++at) {
            while (second ? tile == at && position(tile, u, c) < end : u < U) {
                const int f = first_of(u), cnt = first_of(u + 1) - f;
                const int last = second ? min(nc, c + end - position(tile, u, c)) : nc;
                acc.clear();
#pragma unroll 1
                for (; c < last; ++c) step(cnt);
                float v[4];
                acc.get(v, cnt, lane);
                if (!second) {
                    // The warps' sums meet in one of two buffers; one warp, another for
                    // every tile, adds them up while the rest go on with the next tile.
                    float4 sum = make_float4(v[0], v[1], v[2], v[3]);
                    bool mine = true;
                    if (ks > 1) {
                        const int buf = turn & 1;
                        const uint32_t round = (uint32_t)(turn >> 1) & 1u;
                        float4 *red = s_red + (buf * FW_WARPS + group * ks) * 32 + lane;
                        mbar_wait_bounded(&s_free[group][buf], round ^ 1u, &s_abort);
                        red[(warp & (ks - 1)) * 32] = sum;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_full[group][buf]);
                        mine = (turn & (ks - 1)) == (warp & (ks - 1));
                        if (mine) {
                            mbar_wait_bounded(&s_full[group][buf], round, &s_abort);
                            sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                            for (int w = 0; w < FW_WARPS; ++w) {
                                if (w >= ks) break;
                                const float4 r = red[w * 32];
                                sum.x += r.x;
                                sum.y += r.y;
                                sum.z += r.z;
                                sum.w += r.w;
                            }
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&s_free[group][buf]);
                        }
                        ++turn;
                    }
                    if (mine) {
                        // gate (x, y) and up (z, w) of unit g for the entry's rows 2 q, 2 q + 1
                        const int m = 2 * (lane & 3);
                        T *h = static_cast<T *>(p.h) + (size_t)(f + m) * p.H + tile * 8 + g;
                        T *low = h + (size_t)slots * p.H;
                        if (m < cnt) Elem<T>::put(sum.x / (1.f + expf(-sum.x)) * sum.z, h, low);
                        if (m + 1 < cnt)
                            Elem<T>::put(sum.y / (1.f + expf(-sum.y)) * sum.w, h + p.H, low + p.H);
                    }
                } else {
                    if (SPLIT) {  // columns 4 .. are the second parts' sums
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float low = __shfl_xor_sync(0xffffffffu, v[i], 2);
                            // an infinite weight is infinite by the first part alone: the
                            // second, zero or of the other sign, would make it NaN
                            v[i] = fabsf(v[i]) < INFINITY ? v[i] + low : v[i];
                        }
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int m = 2 * (lane & 3) + half;
                        if (m >= cnt) continue;
                        float *o = s_out + (warp * p.T + s_token[f + m]) * FW_M;
                        const float w = s_w[s_sorted[f + m]];
                        o[g] = fmaf(w, v[half], o[g]);
                        o[g + 8] = fmaf(w, v[2 + half], o[g + 8]);
                    }
                    __syncwarp();
                    if (c < nc) break;  // the part ends here
                }
                c = 0;
                next_segment(tile, u);
            }
            if (!second) continue;
            // the warps' sums; a tile that others share goes through memory
            const bool whole = (at > first_tile || from_start) && (at + 1) * per_tile <= end;
            const int side = at == first_tile ? 0 : 1;
            float *part = p.part + ((size_t)blockIdx.x * 2 + side) * p.T * FW_M;
            if (!whole) cut[side] = at;
            __syncthreads();
            for (int o = tid; o < FW_M * p.T; o += FW_THREADS) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < FW_WARPS; ++w) {
                    sum += s_out[w * FW_M * p.T + o];
                    s_out[w * FW_M * p.T + o] = 0.f;
                }
                const int d = at * FW_M + o % FW_M;
                if (!whole)
                    part[o] = sum;
                else if (d < p.D)
                    out[(size_t)(o / FW_M) * p.D + d] = Elem<T>::round(sum);
            }
            __syncthreads();
        }
        copy_wait<0>();
        __syncthreads();
        if (!second) {
            if (p.phases == FEW_ALL) {
                if (tid == 0) {
                    fence_acq_rel_gpu();
                    red_release_gpu_add(&p.bars[1], 1);
                }
                griddep_launch_dependents();
            }
            continue;
        }
        if (line == 0 || (cut[0] < 0 && cut[1] < 0)) continue;
        // shared tiles: the CTA that comes last adds the parts, in order
        int ca[2], cb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (cut[i] < 0) continue;
            ca[i] = cut_holder(line, G2, cut[i] * per_tile);
            cb[i] = cut_holder(line, G2, (cut[i] + 1) * per_tile - 1);
        }
        if (tid < 2) {
            const int mine = tid == 0 ? cut[0] : cut[1];
            if (mine >= 0) {
                fence_acq_rel_gpu();
                const int from = tid == 0 ? ca[0] : ca[1], others = (tid == 0 ? cb[0] : cb[1]) - from;
                const int shift = 16 * (from & 1);
                const unsigned before = atomicAdd(&p.tile_count[from >> 1], 1u << shift);
                fence_acq_rel_gpu();
                s_last[tid] = (before >> shift & 0xffffu) == (unsigned)others;
                if (s_last[tid]) atomicSub(&p.tile_count[from >> 1], (unsigned)(others + 1) << shift);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (cut[i] < 0 || !s_last[i]) continue;
            for (int o = tid; o < FW_M * p.T; o += FW_THREADS) {
                float sum = 0.f;
                for (int b = ca[i]; b <= cb[i]; ++b) {
                    const int theirs = cut_first(line, G2, b) / per_tile;
                    sum += __ldcg(p.part + ((size_t)b * 2 + (cut[i] == theirs ? 0 : 1)) * p.T * FW_M + o);
                }
                const int d = cut[i] * FW_M + o % FW_M;
                if (d < p.D) out[(size_t)(o / FW_M) * p.D + d] = Elem<T>::round(sum);
            }
        }
    }
    if (U == 0 && !dead && (p.phases & FEW_GEMM2)) {  // no token has an expert here
        T *out = static_cast<T *>(p.out);
        for (long long i = (long long)blockIdx.x * FW_THREADS + tid; i < (long long)p.T * p.D;
             i += (long long)G * FW_THREADS)
            out[i] = Elem<T>::round(0.f);
    }
    copy_wait<0>();
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
                    for (int i = 0; i < kFewMaxCtas / 2; ++i) p.tile_count[i] = 0;
                p.bars[0] = p.bars[1] = p.bars[2] = 0;
            }
        }
    }
}

}  // namespace

// The barriers' counts, polled, on a line of their own, and the tiles': one length
// for all layers, so that what one keeps at zero is not another one's scratch.
constexpr int FW_BARS = 32;
static_assert(kFewMaxCtas % 2 == 0, "two counts to a word");
int few_scratch_ints() { return FW_BARS + kFewMaxCtas / 2; }
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
    p.tile_count = reinterpret_cast<unsigned *>(f.counters + FW_BARS);
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
    // As many steps of every warp as the shared memory takes, one of them being
    // read: 6 for one token (160 KB of weights in flight per SM), 5 for two, else
    // 4 (fp32: 6 to 4), or 3 with many pairs.
    const int rest = few_sum_bytes(f.T) + few_table_bytes(f.T * f.k);
    p.rows = std::min(f.T, f.is_bf16 ? FW_N / 2 : FW_N);
    const int slot = few_slot_bytes(p.rows, f.is_bf16);
    const int depth = std::min(6, (FW_SMEM - rest) / (FW_WARPS * slot));
    const size_t smem = (size_t)FW_WARPS * depth * slot + rest;
    auto fn = f.is_bf16 ? (depth == 6   ? few_layer_kernel<__nv_bfloat16, 6>
                           : depth == 5 ? few_layer_kernel<__nv_bfloat16, 5>
                           : depth == 4 ? few_layer_kernel<__nv_bfloat16, 4>
                                        : few_layer_kernel<__nv_bfloat16, 3>)
                        : (depth == 6   ? few_layer_kernel<float, 6>
                           : depth == 5 ? few_layer_kernel<float, 5>
                           : depth == 4 ? few_layer_kernel<float, 4>
                                        : few_layer_kernel<float, 3>);
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
