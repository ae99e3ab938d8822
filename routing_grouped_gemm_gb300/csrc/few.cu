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
// way, and register accumulators need no TMEM round trip.  A producer warp
// copies row pieces of 1 KB into a ring with bulk copies; a lane takes 16
// consecutive bytes of a row (the sum over k does not care which k meet in one
// instruction, as long as both operands agree), so fragments come straight from
// 16-byte shared loads.  fp32 layers use the same tiles with fused multiply-adds.
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

constexpr int FW_WARPS = 8;  // consumer warps; one more produces
constexpr int FW_THREADS = 32 * (FW_WARPS + 1);
constexpr int FW_CHUNK = 1024;              // bytes of a row in one stage
constexpr int FW_STRIDE = FW_CHUNK + 64;    // two rows' 64-byte pieces cover all banks
constexpr int FW_M = 16;                    // weight rows per tile
constexpr int FW_N = 8;                     // rows of an entry
constexpr int FW_MAX_STAGES = 12;
constexpr int FW_SMEM = 225 * 1024;

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
    int phases, stages;
};

template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float round(float v) { return v; }
};
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
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
    // one 64-byte step of the stage's rows, `off` bytes in; `in`: this lane's 16
    // bytes lie inside the row (else they count as zeros)
    __device__ __forceinline__ void step(const char *a, const char *b, int off, bool in, int cnt,
                                         int lane) {
        const int g = lane >> 2, o = off + (lane & 3) * 16;
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo, bb = lo;
        if (in) {
            lo = *reinterpret_cast<const uint4 *>(a + g * FW_STRIDE + o);
            hi = *reinterpret_cast<const uint4 *>(a + (g + 8) * FW_STRIDE + o);
            // columns past the entry's rows: any row will do, they are not stored
            bb = *reinterpret_cast<const uint4 *>(b + (g < cnt ? g : 0) * FW_STRIDE + o);
        }
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
    __device__ __forceinline__ void step(const char *a, const char *b, int off, bool in, int cnt,
                                         int lane) {
        if (!in) return;
        const int g = lane >> 2, o = off + (lane & 3) * 16;
        const uint4 al = *reinterpret_cast<const uint4 *>(a + g * FW_STRIDE + o);
        const uint4 ah = *reinterpret_cast<const uint4 *>(a + (g + 8) * FW_STRIDE + o);
#pragma unroll
        for (int n = 0; n < FW_N; ++n) {
            if (n >= cnt) break;
            const uint4 bb = *reinterpret_cast<const uint4 *>(b + n * FW_STRIDE + o);
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

// Shared memory behind the ring, in bytes (T k slots, T tokens).
__host__ __device__ inline int few_table_bytes(int slots) { return (slots * 16 + 16 + 15) / 16 * 16; }
__host__ __device__ inline int few_out_bytes(int T) { return FW_WARPS * FW_M * T * 4; }
constexpr int kFewFixed = 2 * FW_WARPS * 32 * 16 /* s_red */ + 2 * FW_MAX_STAGES * 8 + 64;
__host__ __device__ inline int few_stage_bytes(int T) {
    return (FW_M + (T < FW_N ? T : FW_N)) * FW_STRIDE;
}

// Key of expert e for every token, by the CTA's consumer warps.
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
            bar_sync(1, 32 * FW_WARPS);
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
            bar_sync(1, 32 * FW_WARPS);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(FW_THREADS, 1)
few_layer_kernel(const FewParams p) {
    extern __shared__ __align__(128) char smem[];
    __shared__ volatile int s_abort;
    __shared__ int s_local, s_entries, s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = gridDim.x;
    const int slots = p.T * p.k, stage_bytes = few_stage_bytes(p.T);
    char *ring = smem;
    float4 *s_red = reinterpret_cast<float4 *>(ring + p.stages * stage_bytes);  // [2][warps][32]
    uint64_t *full = reinterpret_cast<uint64_t *>(s_red + 2 * FW_WARPS * 32);
    uint64_t *empty = full + FW_MAX_STAGES;
    float *s_out = reinterpret_cast<float *>(empty + FW_MAX_STAGES + 8);  // [warps][T][16]
    float *s_w = s_out + FW_WARPS * FW_M * p.T;                           // [slots]
    int *s_idx = reinterpret_cast<int *>(s_w + slots);                    // [slots], then sorted pairs
    int *s_sorted = s_idx + slots;        // [slots]: slot of the n-th pair in order of (expert, slot)
    uint32_t *s_entry = reinterpret_cast<uint32_t *>(s_sorted + slots);   // [entries + 1]: expert << 16 | first pair
    constexpr int EB = (int)sizeof(T);

    griddep_wait();
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 2);  // the weights' and the rows' bytes are announced apart
            mbar_init(&empty[i], FW_WARPS);
        }
        fence_mbarrier_init();
    }
    __syncthreads();

    // ---- route ----
    if (p.phases & FEW_ROUTE) {
        if (warp < FW_WARPS) few_route<T>(p, reinterpret_cast<float *>(s_red), warp, lane);
        __syncthreads();
        if (p.phases != FEW_ALL) return;
        if (tid == 0) {
            fence_acq_rel_gpu();
            red_release_gpu_add(&p.bars[0], 1);
            wait_count_bounded(&p.bars[0], G, &s_abort);
        }
        __syncthreads();
    }
    const bool dead = s_abort;  // the same for every thread: nothing sets it before the roles part
    // ---- top-k and the entries, every CTA for itself ----
    if (!dead) {
        for (int t = warp; t < p.T; t += FW_WARPS + 1)
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
    const int nt1 = p.H / 8, nc1 = (p.D * EB + FW_CHUNK - 1) / FW_CHUNK;
    const int nt2 = (p.D + FW_M - 1) / FW_M, nc2 = (p.H * EB + FW_CHUNK - 1) / FW_CHUNK;
    const bool do1 = p.phases & FEW_GEMM1, do2 = p.phases & FEW_GEMM2;
    const int tiles1 = do1 ? U * nt1 : 0;
    const long long per_tile = (long long)U * nc2, line = do2 ? per_tile * nt2 : 0;
    // CTAs that take a part of the line: no more than it has chunks, so that none is empty
    const int G2 = (int)min((long long)G, max(line, 1ll));
    const bool part2 = (int)blockIdx.x < G2;
    const long long lo = part2 ? line * blockIdx.x / G2 : 0, hi = part2 ? line * (blockIdx.x + 1) / G2 : 0;
    auto first_of = [&](int u) { return (int)(s_entry[u] & 0xffffu); };

    if (warp == FW_WARPS && !dead) {
        // ---- producer ----
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        auto acquire = [&]() {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[stage], phase ^ 1u, &s_abort));
            return ok;
        };
        auto next = [&]() {
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        };
        auto row_piece = [&](char *dst, const void *base, size_t row, int row_bytes, int c, int bytes,
                             uint64_t *bar) {
            bulk_load(dst, static_cast<const char *>(base) + row * row_bytes + (size_t)c * FW_CHUNK,
                      (uint32_t)bytes, bar);
        };
        for (int i = blockIdx.x; i < tiles1 && ok; i += G) {
            const int u = i / nt1, j = i - u * nt1;
            const int e = s_entry[u] >> 16, f = first_of(u), cnt = first_of(u + 1) - f;
            const int n = lane - FW_M;  // lanes 16 ..: the entry's rows
            const size_t token = n >= 0 && n < cnt ? (size_t)(s_sorted[f + n] / p.k) : 0;
            const size_t row = ((size_t)e * p.H + (size_t)j * 8 + (lane & 7));
            for (int c = 0; c < nc1 && acquire(); ++c, next()) {
                const int bytes = min(FW_CHUNK, p.D * EB - c * FW_CHUNK);
                char *st = ring + stage * stage_bytes;
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], FW_M * bytes);
                if (lane == FW_M) mbar_arrive_expect_tx(&full[stage], cnt * bytes);
                __syncwarp();
                if (lane < FW_M)
                    row_piece(st + lane * FW_STRIDE, lane < 8 ? p.w1 : p.w3, row, p.D * EB, c, bytes,
                              &full[stage]);
                else if (n < cnt)
                    row_piece(st + lane * FW_STRIDE, p.x, token, p.D * EB, c, bytes, &full[stage]);
            }
        }
        // GEMM2: the weights' part of the first stages goes out before the
        // barrier, the rows' part (h) behind it
        auto place = [&](long long i, int *dt, int *u, int *c) {
            *dt = (int)(i / per_tile);
            const int r = (int)(i - (long long)*dt * per_tile);
            *u = r / nc2;
            *c = r - *u * nc2;
        };
        auto load_w2 = [&](long long i) {
            int dt, u, c;
            place(i, &dt, &u, &c);
            const int e = s_entry[u] >> 16, rows = min(FW_M, p.D - dt * FW_M);
            const int bytes = min(FW_CHUNK, p.H * EB - c * FW_CHUNK);
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], rows * bytes);
            __syncwarp();
            if (lane < rows)
                row_piece(ring + stage * stage_bytes + lane * FW_STRIDE, p.w2,
                          (size_t)e * p.D + (size_t)dt * FW_M + lane, p.H * EB, c, bytes, &full[stage]);
        };
        auto load_h = [&](long long i) {
            int dt, u, c;
            place(i, &dt, &u, &c);
            const int f = first_of(u), cnt = first_of(u + 1) - f;
            const int bytes = min(FW_CHUNK, p.H * EB - c * FW_CHUNK);
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], cnt * bytes);
            __syncwarp();
            if (lane < cnt)
                row_piece(ring + stage * stage_bytes + (FW_M + lane) * FW_STRIDE, p.h, (size_t)(f + lane),
                          p.H * EB, c, bytes, &full[stage]);
        };
        if (ok && do2) {
            const int stage0 = stage;
            const uint32_t phase0 = phase;
            const int ahead = (int)min((long long)p.stages, hi - lo);
            for (int i = 0; i < ahead && acquire(); ++i, next()) load_w2(lo + i);
            if (ok && p.phases == FEW_ALL) {
                bool there = true;
                if (lane == 0) there = wait_count_bounded(&p.bars[1], G, &s_abort);
                ok = __all_sync(0xffffffffu, there);
            }
            if (ok) {
                __syncwarp();
                fence_proxy_async_global();  // h was written by ordinary stores
                stage = stage0;
                phase = phase0;
                for (int i = 0; i < ahead; ++i, next()) load_h(lo + i);
                for (long long i = lo + ahead; i < hi && acquire(); ++i, next()) {
                    load_w2(i);
                    load_h(i);
                }
            }
        }
    } else if (!dead) {
        // ---- consumers ----
        int stage = 0, turn = 0;
        uint32_t phase = 0;
        Acc<T> acc;
        // one stage: the row pieces' 64-byte steps, this warp's every eighth
        auto consume = [&](int bytes, int cnt) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[stage], phase, &s_abort))) return false;
            const char *a = ring + stage * stage_bytes, *b = a + FW_M * FW_STRIDE;
#pragma unroll
            for (int i = 0; i < FW_CHUNK / 64 / FW_WARPS; ++i) {
                const int off = (warp + i * FW_WARPS) * 64;
                if (off < bytes) acc.step(a, b, off, off + (lane & 3) * 16 < bytes, cnt, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == p.stages) { stage = 0; phase ^= 1u; }
            return true;
        };
        bool ok = true;
        for (int i = blockIdx.x; i < tiles1 && ok; i += G) {
            const int u = i / nt1, j = i - u * nt1;
            const int f = first_of(u), cnt = first_of(u + 1) - f;
            acc.clear();
            for (int c = 0; c < nc1 && ok; ++c) ok = consume(min(FW_CHUNK, p.D * EB - c * FW_CHUNK), cnt);
            float v[4];
            acc.get(v, lane);
            float4 *red = s_red + turn * FW_WARPS * 32;
            turn ^= 1;  // the other buffer's readers are behind the barrier before this one
            red[warp * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
            ok = bar_and(1, 32 * FW_WARPS, ok);
            if (ok && tid < 64) {
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
                    static_cast<T *>(p.h)[(size_t)(f + n) * p.H + j * 8 + (lane >> 2)] =
                        Elem<T>::round(gate / (1.f + expf(-gate)) * up);
            }
        }
        if (do1 && p.phases == FEW_ALL) {
            // h is read by the other CTAs' bulk copies
            fence_proxy_async_global();
            ok = bar_and(1, 32 * FW_WARPS, ok);
            if (tid == 0) {
                fence_acq_rel_gpu();
                red_release_gpu_add(&p.bars[1], 1);
            }
            griddep_launch_dependents();
        }
        if (do2 && ok) {
            for (int i = lane; i < FW_M * p.T; i += 32) s_out[warp * FW_M * p.T + i] = 0.f;
            __syncwarp();
            const int first_dt = per_tile ? (int)(lo / per_tile) : 0;
            for (long long i = lo; i < hi && ok;) {
                const int dt = (int)(i / per_tile);
                const long long end = min(hi, (long long)(dt + 1) * per_tile);
                const bool whole = i == (long long)dt * per_tile && end == i + per_tile;
                while (i < end && ok) {  // this CTA's part of one entry
                    const int r = (int)(i - (long long)dt * per_tile), u = r / nc2;
                    int c = r - u * nc2;
                    const int f = first_of(u), cnt = first_of(u + 1) - f;
                    acc.clear();
                    for (; c < nc2 && i < end && ok; ++c, ++i)
                        ok = consume(min(FW_CHUNK, p.H * EB - c * FW_CHUNK), cnt);
                    float v[4];
                    acc.get(v, lane);
                    const int g = lane >> 2;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int n = 2 * (lane & 3) + half;
                        if (n >= cnt) continue;
                        const int slot = s_sorted[f + n];
                        float *o = s_out + (warp * p.T + slot / p.k) * FW_M;
                        o[g] = fmaf(s_w[slot], v[half], o[g]);
                        o[g + 8] = fmaf(s_w[slot], v[2 + half], o[g + 8]);
                    }
                }
                ok = bar_and(1, 32 * FW_WARPS, ok);
                if (!ok) break;
                // the warps' sums; a tile that others share goes through memory
                float *part = p.part + ((size_t)blockIdx.x * 2 + (dt == first_dt ? 0 : 1)) * p.T * FW_M;
                T *out = static_cast<T *>(p.out);
                for (int o = tid; o < FW_M * p.T; o += 32 * FW_WARPS) {
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
                bar_sync(1, 32 * FW_WARPS);
                if (whole) continue;
                // CTAs that share the tile: c0 .. c1
                const long long a0 = (long long)dt * per_tile, a1 = a0 + per_tile;
                int c0 = (int)(a0 * G2 / line), c1 = (int)min((long long)G2 - 1, (a1 - 1) * G2 / line);
                while (line * (c0 + 1) / G2 <= a0) ++c0;
                while (c0 > 0 && line * c0 / G2 > a0) --c0;
                while (line * (c1 + 1) / G2 < a1) ++c1;
                while (c1 > 0 && line * c1 / G2 >= a1) --c1;
                if (tid == 0) {
                    fence_acq_rel_gpu();
                    const int before = atomicAdd(&p.tile_count[dt], 1);
                    fence_acq_rel_gpu();
                    s_last = before == c1 - c0;
                    if (s_last) p.tile_count[dt] = 0;
                }
                bar_sync(1, 32 * FW_WARPS);
                if (s_last)
                    for (int o = tid; o < FW_M * p.T; o += 32 * FW_WARPS) {
                        float sum = 0.f;
                        for (int c = c0; c <= c1; ++c) {
                            const int theirs = (int)(line * c / G2 / per_tile);
                            sum += __ldcg(p.part + ((size_t)c * 2 + (dt == theirs ? 0 : 1)) * p.T * FW_M + o);
                        }
                        const int d = dt * FW_M + o % FW_M;
                        if (d < p.D) out[(size_t)(o / FW_M) * p.D + d] = Elem<T>::round(sum);
                    }
                bar_sync(1, 32 * FW_WARPS);  // s_last is free again
            }
            if (line == 0) {  // no token has an expert here
                T *out = static_cast<T *>(p.out);
                for (long long i = (long long)blockIdx.x * 32 * FW_WARPS + tid; i < (long long)p.T * p.D;
                     i += (long long)G * 32 * FW_WARPS)
                    out[i] = Elem<T>::round(0.f);
            }
        }
    }
    __syncthreads();
    const bool aborted = s_abort;
    if (aborted) {
        if (warp == 0) settle_inflight_copies();
        __syncthreads();
    }
    if (tid == 0) {
        if (aborted) raise_flag(p.status, FLAG_TIMEOUT);
        if (p.phases == FEW_ALL) {
            // the last CTA to leave puts the counters back
            fence_acq_rel_gpu();
            if (atomicAdd(&p.bars[2], 1) == G - 1) {
                fence_acq_rel_gpu();
                const int late = atomicOr(p.status, 0) & FLAG_TIMEOUT;
                if (late)  // some parts never came
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
    const int rest = kFewFixed + few_out_bytes(f.T) + few_table_bytes(f.T * f.k);
    p.stages = std::min(FW_MAX_STAGES, (FW_SMEM - rest) / few_stage_bytes(f.T));
    const size_t smem = (size_t)p.stages * few_stage_bytes(f.T) + rest;
    const void *kernel = f.is_bf16 ? (const void *)few_layer_kernel<__nv_bfloat16>
                                   : (const void *)few_layer_kernel<float>;
    cudaError_t err = ensure_smem(kernel, smem);
    if (err != cudaSuccess) return err;
    const int ctas = std::min(sm_count(), kFewMaxCtas);
    if (ctas <= 0) return cudaErrorInvalidDevice;
    auto fn = f.is_bf16 ? few_layer_kernel<__nv_bfloat16> : few_layer_kernel<float>;
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
