// MXFP4 m-grouped SwiGLU expert FFN on CTA pairs (tcgen05 kind::mxf4, block
// scales).
//
// Same contract as grouped_tc.cu over operands of e2m1 codes with one e8m0
// scale per 32 elements of K (mxfp4_row.cuh):
//   g = sum_b 2^(ex[r,b] + e1[n,b]) sum_{i in b} qx[r,i] q1[n,i],  u with w3,
//   h = mxfp4(SiLU(g) u),  y = fp16(h w2^T).
// Products of codes are exact, the tensor cores apply the scales and sum in
// fp32; h is rounded once, from the fp32 result straight to MXFP4 (GEMM2's
// operand), and y once to fp16, as the other bf16 layers store it.
//
// At 4 bits the tensor cores take a K = 64 step in the time of a bf16 K = 16
// one, so everything around them counts.  Decode calls run at the weights' HBM
// time (256 experts' 5.9 GB in 854 us).  A prompt of a few hundred rows per expert
// (4096 tokens x 6, 64 experts of 2048 x 1408: 113 us, 3.8 PFLOP/s) has the tensor
// pipe busy 45% of GEMM1 and 37% of GEMM2: about 14 us are the launches'
// beginnings, the epilogue took 22 of 122 us when it was left out, operands and
// scales from L2 up to 2 us each.  A long Zipf-skewed one (16384 tokens x 8, 64
// experts of 4096 x 1536) takes 826 us, 6.0 PFLOP/s: 80% of four times the bf16
// rate measured on the GPU.  So, few operand rows per product:
//   * the weights are the M operand, 256 rows on a pair of CTAs
//     (cta_group::2), and the tokens the N operand, up to 32, 144 or 208 of an
//     expert's rows (the launch says when which), split evenly over its tiles in
//     steps of 16: a ragged segment costs its own rows and no more, a decode
//     batch loads 16;
//   * of GEMM1's 256 rows each CTA holds 64 rows of w1 and the same 64 of w3,
//     so a tile gives h of 128 hidden units;
//   * two accumulators leave at least 96 of the 512 tensor-memory columns for
//     scales: four or more buffers of 24 (a K block of 256 of 128 weight rows
//     and of the tokens), taken in turn.  The warp that copies scales refills one
//     when the MMAs that many K blocks back have completed, which the ring's own
//     barriers tell, so the buffers and the stages differ in number freely;
//   * scales are read in their natural [rows, K / 32] layout, which is not the
//     order the tensor cores want (four scales each of rows l, l + 32, l + 64
//     and l + 96 together).  Warps fetch them, 32 bytes of a row -- one
//     sector, four K blocks -- at a time, and store them as 512-byte blocks for
//     tcgen05.cp, in a ring of their own with one fence and one arrival for four
//     K blocks;
//   * the accumulator's lanes are weight rows and its columns tokens, so the
//     epilogues turn it around in shared memory, 16 or 32 tokens at a time: for
//     h a thread then has 8 or 16 gates and ups of one token (part of a block,
//     its maximum one or two shuffles away), for y pieces of a token's row;
//   * every mbarrier wait is bounded (FLAG_TIMEOUT).
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "launch.h"
#include "mxfp4_row.cuh"

namespace moe {
namespace {

constexpr int X_BM = 256;             // weight rows per pair tile, 128 per CTA
constexpr int X_UNITS = X_BM / 2;     // hidden units per GEMM1 tile
constexpr int X_BK = 256;             // K elements per stage
constexpr int X_ROW = X_BK / 2;       // bytes of a row's K block: the swizzle span
constexpr int X_W_BYTES = 128 * X_ROW;
constexpr int X_SF_BLOCK = 512;       // 128 rows x 4 scales
constexpr int X_SF_BYTES = 6 * X_SF_BLOCK;  // two K halves of the weights' block, then of the tokens' two
constexpr int X_MAX_STAGES = 8;
constexpr int X_GROUP = 4;            // K blocks whose scales are fetched together (32 bytes of a row)
constexpr int X_GROUP_BYTES = X_GROUP * X_SF_BYTES;
constexpr int X_SLOTS = 2;            // groups in shared memory
constexpr int X_SF_WARPS = 2 * X_SLOTS;  // per slot one for the weights' scales, one for the tokens'
// Warps: TMA, MMA, scale copies, scale fetchers, epilogue.
constexpr int X_EPI_GROUPS = 2;       // of four warps (the TMEM lane quarters), taking chunks of a tile in turn
constexpr int X_EPI_WARPS = 4 * X_EPI_GROUPS;
constexpr int X_THREADS = 32 * (3 + X_SF_WARPS + X_EPI_WARPS);
constexpr int X_TMEM_COLS = 512;
constexpr int X_SF_COLS = 24;         // of a K block: 2 x 4 of the weights, 2 x 8 of the tokens
constexpr int X_NBARS = 2 * X_MAX_STAGES + 2 * X_SLOTS + 6;
constexpr int X_SMEM_MAX = 227 * 1024;
constexpr int X_TURN_LD = 132;        // GEMM1's turning buffer: a token's 64 gates, 64 ups, 4 of padding
constexpr int X_TURN2 = X_EPI_WARPS * 32 * 64;  // GEMM2's: per warp 32 tokens x 32 columns fp16
constexpr int X_EPI_BAR = 1;          // named barriers of the epilogue: one per group

// What follows from the most tokens of a tile, kBN (a multiple of 16).
template <int kBN>
struct MxShape {
    static constexpr int kTBytes = kBN / 2 * X_ROW;         // a CTA's tokens of a stage
    static constexpr int kStage = X_W_BYTES + kTBytes;
    static constexpr int kSfCol = 2 * kBN;                  // scale buffers start behind two accumulators
    static constexpr int kSfBufs = (X_TMEM_COLS - kSfCol) / X_SF_COLS;
    // tokens that an epilogue group of GEMM1 turns around at a time: 16 where
    // calls wait for weights and the room is better spent on two more stages
    static constexpr int kChunk1 = kBN > 144 ? 32 : 16;
    static constexpr int kTurn1 = X_EPI_GROUPS * kChunk1 * X_TURN_LD * 4;
    static_assert(kBN % 16 == 0 && kBN <= 256 && kTBytes % 1024 == 0 && kSfBufs >= 2, "tile shape");
};

struct MxParams {
    int E_local, e_first, rows_alloc;
    int stages;           // of the ring
    int K, nk;            // reduction length (D or H_local) and its 256-blocks
    int nt, n_out;        // tiles along the weight rows; columns of the output (H_local or D)
    const int *seg_off, *tpe;
    const uint8_t *t_sf;          // tokens' scales [rows_alloc, K / 32]
    const uint8_t *w_sf0, *w_sf1; // of w1 and w3 [E_local, H_local, D / 32], or of w2 twice
    uint8_t *hq, *hsf;            // GEMM1: codes [rows, H / 2], scales [rows, H / 32]
    __half *y;                    // GEMM2: [rows, D]
    int *status;
};

template <bool kGemm1, int kBN>
size_t mx_smem_bytes(int stages, int E_local) {
    return 1024 + (size_t)stages * MxShape<kBN>::kStage + X_SLOTS * X_GROUP_BYTES +
           (kGemm1 ? MxShape<kBN>::kTurn1 : X_TURN2) + (X_NBARS + 1) * sizeof(uint64_t) + 16 +
           sizeof(int) * (4 * (size_t)E_local + 1);
}

// The experts' rows in shared memory: first row, rows, first token tile and
// rows per token tile.
struct MxTable {
    int *base, *valid, *first, *per;
};

// A warp's way through the tiles of its pair: tile v = token tile * nt +
// weight tile, an expert's rows in equal token tiles (a multiple of 16, at
// most kBN), weight tiles inner.  Every step is n_pairs tiles on, so a few
// additions and the next experts' entries replace a division and a search.
struct MxTile {
    int tt, nt;                    // token tile (over all experts), weight tile
    int expert, row0, nvalid;      // expert, first row, rows
    int n;                         // the MMA's N: nvalid rounded up to 16

    __device__ __forceinline__ void place(const MxTable &t) {
        while (t.first[expert + 1] <= tt) ++expert;
        const int per = t.per[expert], lead = (tt - t.first[expert]) * per;
        row0 = t.base[expert] + lead;
        nvalid = min(per, t.valid[expert] - lead);
        n = (nvalid + 15) & ~15;
    }
    __device__ __forceinline__ MxTile(int v, int nts, int total, const MxTable &t)
        : tt(v / nts), nt(v - v / nts * nts), expert(0), row0(0), nvalid(0), n(16) {
        if (v < total) place(t);
    }
    // n_pairs on, in units of token tiles (dt) and weight tiles (dn)
    __device__ __forceinline__ void step(int dt, int dn, int nts, bool more, const MxTable &t) {
        tt += dt;
        nt += dn;
        if (nt >= nts) {
            nt -= nts;
            ++tt;
        }
        if (more) place(t);
    }
};

// An expert's first row, rows and token tiles (kept in `first` until the scan),
// by every warp but the scale fetchers, so that E_local = 256 waits for one load
// and not for eight in a row.
// Offsets outside [0, rows_alloc] or decreasing flag FLAG_BAD_ROUTING and empty
// the segment.
template <int kBN>
__device__ __forceinline__ void read_mx_table(const MxParams &p, const MxTable &t, int *status) {
    const int warp = threadIdx.x >> 5;
    const int first = threadIdx.x - (warp < 3 ? 0 : 32 * X_SF_WARPS);
    for (int e = first; e < p.E_local; e += X_THREADS - 32 * X_SF_WARPS) {
        const int b = p.seg_off[e], end = p.seg_off[e + 1];
        int c = p.tpe[p.e_first + e];
        if (b < 0 || end < b || end > p.rows_alloc || c < 0) {
            raise_flag(status, FLAG_BAD_ROUTING);
            c = 0;
        }
        const int v = max(0, min(c, end - b));
        const int tiles = (v + kBN - 1) / kBN;
        t.base[e] = b;
        t.valid[e] = v;
        t.first[e] = tiles;
        t.per[e] = tiles ? ((v + tiles - 1) / tiles + 15) & ~15 : 16;
    }
}

// Exclusive scan of the tile counts by one warp.
__device__ __forceinline__ void scan_mx_table(int lane, int E_local, const MxTable &t) {
    int run = 0;
    for (int e0 = 0; e0 < E_local; e0 += 32) {
        const int e = e0 + lane;
        const int tiles = e < E_local ? t.first[e] : 0;
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += n;
        }
        if (e < E_local) t.first[e] = run + incl - tiles;
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) t.first[E_local] = run;
}

// SiLU(g) = g / (1 + e^-g), as g e^g / (1 + e^g) below zero: the divisor stays in
// [1, 2], and the result keeps its value where e^-g would leave fp32's range, for g
// from -87 down.  e^-|g| is taken 2^24 times as large, as an ordinary number down to
// fp32's smallest (2^-149).  The exponent's rounding is the largest error: 2^-21 for
// small gates, 2^-18 at |g| = 100, far below the 4-bit rounding.  (As fast as
// g / (1 + e^-g) with the fast exponential and division; those with this split cost
// fine-grained 115.4 against 113.3 us.)
__device__ __forceinline__ float mx_silu(float g) {
    const float t24 = ex2_approx(fmaf(fabsf(g), -1.44269504f, 24.f));
    const float r = rcp_approx(fmaf(t24, 0x1p-24f, 1.f));
    return (g < 0.f ? g * (t24 * 0x1p-24f) : g) * r;
}

constexpr uint32_t kMxOnes = 0x7f7f7f7fu;  // four scales of 1

// Bytes [32 kg, 32 kg + 32) of each of N rows of scales [.., ld], ld a multiple
// of 4 (the array 16-byte aligned); 1.0 past the row's end (the codes there are
// zeros) and for a row that is not `there`.  The rows' alignment is looked at
// once, not row by row, so that every load is issued before any is used.  Every
// lane reads a row of its own, 32 lines a load, so what counts is how many loads
// a row takes: one where rows lie on 32 bytes (two of 16: Zipf-skewed grouped
// call 829 against 816 us, 256 experts 1263 against 1245).
template <int N>
__device__ __forceinline__ void load_scales32(const uint8_t *const (&base)[N], const size_t (&row)[N],
                                              const bool (&there)[N], int ld, int kg,
                                              uint32_t (&v)[N][8]) {
    const int n = ld - 32 * kg;  // bytes left in a row
    if ((ld & 31) == 0 && (reinterpret_cast<uintptr_t>(base[0]) & 31) == 0 &&
        (reinterpret_cast<uintptr_t>(base[N - 1]) & 31) == 0) {
#pragma unroll
        for (int r = 0; r < N; ++r) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][i] = kMxOnes;
            if (there[r]) ld_global_32(base[r] + row[r] * ld + 32 * kg, v[r]);
        }
        return;
    }
    if ((ld & 15) == 0) {
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const uint4 *q = reinterpret_cast<const uint4 *>(base[r] + row[r] * ld + 32 * kg);
            uint4 a = make_uint4(kMxOnes, kMxOnes, kMxOnes, kMxOnes), b = a;
            if (there[r]) a = q[0];
            if (there[r] && n > 16) b = q[1];
            v[r][0] = a.x; v[r][1] = a.y; v[r][2] = a.z; v[r][3] = a.w;
            v[r][4] = b.x; v[r][5] = b.y; v[r][6] = b.z; v[r][7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int r = 0; r < N; ++r) {
        const uint32_t *q = reinterpret_cast<const uint32_t *>(base[r] + row[r] * ld + 32 * kg);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t x = kMxOnes;
            if (there[r] && 4 * i < n) x = q[i];
            v[r][i] = x;
        }
    }
}

// What a scale warp works with: its room in shared memory, the barriers of that
// and its place among the pair's tiles.
struct ScaleWarp {
    uint8_t *room;
    uint64_t *empty;
    uint32_t full_leader;
    volatile int *abort_flag;
    int slot, lane, pair_id, n_pairs, dt, dn, rank;
};

// Takes every X_SLOTS-th group of four K blocks: 32 bytes of each of the CTA's
// 128 weight rows, or of the tile's tokens (all of them: each CTA's half of the
// MMA needs all).  Lane l serves rows l, l + 32, ...  A group's loads are issued
// when the warp's last one is stored.
// The first round is a dry one, before the wait for the previous kernel and the
// table: no row is there and nothing is announced, but its instructions come from
// memory while there is nothing else to do.  Between the table and the first MMA
// of a fine-grained GEMM2 lay 6.6 us, 3 of them for the instructions up to the
// loads, and for rows at any byte, unrolled, 13 (grouped call 119.8 against 117
// us with the dry round, 37 against 27 for a small shard of such rows).
// kWords: ld is a multiple of 4.
template <bool kGemm1, bool kTokens, int kBN, bool kWords>
__device__ __forceinline__ void fetch_scales(const ScaleWarp &f, const MxParams &p, const MxTable &table) {
    constexpr int kRows = kTokens ? (kBN + 31) / 32 : 4;
    static_assert(kRows <= 8, "two blocks of 128 tokens");
    const int lane = f.lane, ld = p.K / 32, ng = (p.nk + X_GROUP - 1) / X_GROUP;
    const size_t all = (kTokens ? (size_t)p.rows_alloc : (size_t)p.E_local * p.n_out) * ld;
    uint32_t ph = 0, tail = 0;  // tail: the array's last word, where that is a part of one
    MxTile c(f.pair_id, p.nt, 0, table);
    int kg = f.slot, tile = f.pair_id, total = 0;
    int rows_there = 0;  // of the weights (no token is in a tile without rows)
    int dry;
    asm volatile("mov.s32 %0, 1;" : "=r"(dry));  // unknown to the compiler: one code for all rounds
    for (;;) {
        if (!dry) {
            while (kg >= ng && tile < total) {
                kg -= ng;
                tile += f.n_pairs;
                c.step(f.dt, f.dn, p.nt, tile < total, table);
            }
            if (tile >= total) break;
        }
        const uint8_t *base[kRows];
        size_t row[kRows];
        bool there[kRows];
        uint32_t v[kRows][8];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (kTokens) {
                const int r = i * 32 + lane;
                there[i] = r < c.nvalid;
                base[i] = p.t_sf;
                row[i] = (size_t)(c.row0 + r);
            } else {
                const int r = kGemm1 ? c.nt * X_UNITS + f.rank * 64 + (i & 1) * 32 + lane
                                     : c.nt * X_BM + f.rank * 128 + i * 32 + lane;
                there[i] = r < rows_there;
                base[i] = kGemm1 && i >= 2 ? p.w_sf1 : p.w_sf0;
                row[i] = (size_t)c.expert * p.n_out + r;
            }
        }
        // rows at any byte: the aligned words around the 32 bytes, shifted; the
        // first are asked for here, and bring most of the others' sectors
        auto word = [&](int i, int at) {
            const size_t a = ((row[i] * ld + 32 * kg) & ~(size_t)3) + 4 * at;
            const int end = (int)((row[i] * ld) & 3) + min(ld - 32 * kg, 32);
            if (!there[i] || 4 * at >= end) return 0u;
            return a + 4 <= all ? *reinterpret_cast<const uint32_t *>(base[i] + a) : tail;
        };
        if constexpr (kWords) {
            load_scales32<kRows>(base, row, there, ld, kg, v);
        } else {
#pragma unroll
            for (int i = 0; i < kRows; ++i) v[i][0] = word(i, 0);
        }
        if (!dry) {
            // lane 0 waits for the group's room, the warp follows it
            bool got = true;
            if (lane == 0) got = mbar_wait_bounded(f.empty, ph ^ 1u, f.abort_flag);
            if (!__shfl_sync(0xffffffffu, got, 0)) break;
            ph ^= 1u;
        }
        // K block j / 2 of the group, its half h = j % 2, in blocks of 512 bytes:
        // 0, 1: the weights' K halves; 2 + 2 h + token / 128: the tokens'
        auto store = [&](int j, auto &&of) {
            uint4 *d = reinterpret_cast<uint4 *>(f.room + (j / 2) * X_SF_BYTES) + lane;
            const int h = j & 1;
            if constexpr (kTokens) {
                d[32 * (2 + 2 * h)] = make_uint4(of(0), of(1), of(2), of(3));
                if (kBN > 128 && c.n > 128)
                    d[32 * (3 + 2 * h)] = make_uint4(of(4), of(5), of(6), of(7));
            } else {
                d[32 * h] = make_uint4(of(0), of(1), of(2), of(3));
            }
        };
        if constexpr (kWords) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                store(j, [&](int i) { return i < kRows ? v[i < kRows ? i : 0][j] : kMxOnes; });
        } else {
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                const int left = ld - 32 * kg - 4 * j;  // bytes of the row from here on
                const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const uint32_t next = word(i, j + 1);
                    v[i][1] = __funnelshift_r(v[i][0], next, 8 * (uint32_t)((row[i] * ld) & 3));
                    v[i][1] = there[i] ? (v[i][1] & keep) | (kMxOnes & ~keep) : kMxOnes;
                    v[i][0] = next;
                }
                store(j, [&](int i) { return i < kRows ? v[i < kRows ? i : 0][1] : kMxOnes; });
            }
        }
        if (dry) {
            dry = 0;
            bar_sync(0, X_THREADS);  // the table is read
            bar_sync(0, X_THREADS);  // and scanned
            total = table.first[p.E_local] * p.nt;
            if (tile < total) c.place(table);
            griddep_wait();          // every input of this kernel is complete
            rows_there = p.n_out;
            if (!kWords && kTokens && (all & 3)) {
                const size_t a = all & ~(size_t)3;
                for (int i = 0; i < (int)(all & 3); ++i) tail |= (uint32_t)p.t_sf[a + i] << (8 * i);
            }
            continue;
        }
        // tcgen05.cp, issued by the leader's copy warp, reads them through the async
        // proxy; the leader acquires at cluster scope
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            fence_release_smem_cluster();
            mbar_arrive_cluster_relaxed(f.full_leader);
        }
        kg += X_SLOTS;
    }
}

template <bool kGemm1, int kBN>
__global__ void __launch_bounds__(X_THREADS, 1)
grouped_mx_kernel(const __grid_constant__ CUtensorMap tmT8, const __grid_constant__ CUtensorMap tmT16,
                  const __grid_constant__ CUtensorMap tmT32, const __grid_constant__ CUtensorMap tmT64,
                  const __grid_constant__ CUtensorMap tmW0, const __grid_constant__ CUtensorMap tmW1,
                  const MxParams p) {
    // The next kernel may be scheduled now; GEMM2 once GEMM1's inputs are complete,
    // so that it can read the experts' table, one of them, before its own wait.
    if (!kGemm1) griddep_launch_dependents();
    if (cluster_nctarank() != 2) {  // every role below assumes a CTA pair
        griddep_wait();
        if (threadIdx.x == 0) raise_flag(p.status, FLAG_LAUNCH);
        return;
    }
    using Shape = MxShape<kBN>;
    const int stages = p.stages;
    const int sf_bufs = min(Shape::kSfBufs, stages);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sfs = ring + stages * Shape::kStage;  // [X_SLOTS] groups of scales
    uint8_t *turn = sfs + X_SLOTS * X_GROUP_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(turn + (kGemm1 ? Shape::kTurn1 : X_TURN2));
    uint64_t *full = bars;                       // leader: both CTAs' TMA bytes, scales in TMEM -> MMA
    uint64_t *empty = bars + X_MAX_STAGES;       // MMA -> each CTA's TMA, the leader's scale copies
    uint64_t *tfull = bars + 2 * X_MAX_STAGES;   // [2] MMA -> each CTA's epilogue
    uint64_t *tempty = tfull + 2;                // [2] leader: both epilogues -> MMA
    uint64_t *drain = tempty + 2;                // [2] leader: MMA's and copies' completion at exit
    uint64_t *sfull = drain + 2;                 // [X_SLOTS] leader: both CTAs' group of scales -> copies
    uint64_t *sempty = sfull + X_SLOTS;          // [X_SLOTS] copies -> each CTA's scale warp
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + X_NBARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    MxTable table;
    table.base = reinterpret_cast<int *>(tmem_slot + 4);
    table.valid = table.base + p.E_local;
    table.per = table.valid + p.E_local;
    table.first = table.per + p.E_local;  // [E_local + 1]

    // warp-uniform for the compiler too
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair_id = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
    // barriers and tensor memory need no input: ready before the wait for the
    // previous kernel, the table after it
    if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < stages; ++s) {
                mbar_init(&full[s], 2);
                mbar_init(&empty[s], 1);
            }
            for (int a = 0; a < 2; ++a) {
                mbar_init(&tfull[a], 1);
                mbar_init(&tempty[a], 2 * X_EPI_WARPS);
                mbar_init(&drain[a], 1);
            }
            for (int g = 0; g < X_SLOTS; ++g) {
                mbar_init(&sfull[g], 4);  // two warps of each CTA
                mbar_init(&sempty[g], 1);
            }
            *abort_flag = 0;
            fence_mbarrier_init();
        }
        __syncwarp();
    } else if (warp == 2) {
        tmem_alloc_pair(tmem_slot, X_TMEM_COLS);
        tmem_relinquish_pair();
    } else if (warp == 3 && lane == 0) {
        prefetch_tmap(&tmT8);
        prefetch_tmap(&tmT16);
        prefetch_tmap(&tmT32);
        prefetch_tmap(&tmT64);
        prefetch_tmap(&tmW0);
        if (kGemm1) prefetch_tmap(&tmW1);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers exist before anything arrives on them
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int dt = n_pairs / p.nt, dn = n_pairs - dt * p.nt;  // a step of n_pairs tiles
    int total = 0;
    if (warp < 3 || warp >= 3 + X_SF_WARPS) {  // (the scale fetchers: after their dry round)
        if (kGemm1) {
            griddep_wait();  // every input of this kernel is complete
            griddep_launch_dependents();
        }
        read_mx_table<kBN>(p, table, blockIdx.x == 0 ? p.status : nullptr);
        bar_sync(0, X_THREADS);
        if (warp == 0) scan_mx_table(lane, p.E_local, table);
        bar_sync(0, X_THREADS);
        total = table.first[p.E_local] * p.nt;
    }
    const uint32_t full_leader = mapa_shared(smem_u32(&full[0]), 0);

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        // the whole warp walks the tiles and waits, one lane issues
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        MxTile c(pair_id, p.nt, total, table);
        if (!kGemm1) griddep_wait();  // h is complete
        for (int tile = pair_id; ok && tile < total;) {
            const int trows = c.n / 2;  // this CTA's token rows: a multiple of 8, below 128
            const int trow = c.row0 + (int)rank * trows;
            const int wrow = kGemm1 ? c.nt * X_UNITS + (int)rank * 64 : c.nt * X_BM + (int)rank * 128;
            const uint32_t tx = 2u * (uint32_t)(X_W_BYTES + trows * X_ROW);
            for (int kb = 0; kb < p.nk; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], ph ^ 1u, abort_flag))) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    if (leader) mbar_arrive_expect_tx(&full[s], tx);
                    uint8_t *sw = ring + s * Shape::kStage;
                    uint8_t *st = sw + X_W_BYTES;
                    const uint32_t fb = full_leader + (uint32_t)(s * sizeof(uint64_t));
                    tma_load_3d_pair(sw, &tmW0, fb, kb * X_ROW, wrow, c.expert);
                    if (kGemm1)
                        tma_load_3d_pair(sw + X_W_BYTES / 2, &tmW1, fb, kb * X_ROW, wrow, c.expert);
                    int at = 0;
                    if (trows & 64) {
                        tma_load_2d_pair(st, &tmT64, fb, kb * X_ROW, trow);
                        at = 64;
                    }
                    if (trows & 32) {
                        tma_load_2d_pair(st + at * X_ROW, &tmT32, fb, kb * X_ROW, trow + at);
                        at += 32;
                    }
                    if (trows & 16) {
                        tma_load_2d_pair(st + at * X_ROW, &tmT16, fb, kb * X_ROW, trow + at);
                        at += 16;
                    }
                    if (trows & 8)
                        tma_load_2d_pair(st + at * X_ROW, &tmT8, fb, kb * X_ROW, trow + at);
                }
                __syncwarp();
                if (++s == stages) { s = 0; ph ^= 1u; }
            }
            tile += n_pairs;
            c.step(dt, dn, p.nt, tile < total, table);
        }
    } else if (warp == 1) {
        if (leader) {
            // ---------------- MMA issuer (leader CTA) ----------------
            int s = 0, sb = 0;  // stage, scale buffer
            uint32_t ph = 0;
            bool ok = true;
            int it = 0;
            const uint64_t w_desc0 = sdesc_kmajor_sw128(smem_u32(ring));
            MxTile c(pair_id, p.nt, total, table);
            for (int tile = pair_id; ok && tile < total; ++it) {
                const int acc = it & 1;
                const uint32_t id0 = idesc_mxf4_f32(X_BM, c.n, 0), id2 = idesc_mxf4_f32(X_BM, c.n, 2);
                // the peer's epilogue arrives here too: at cluster scope
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(&tempty[acc], ((uint32_t)(it >> 1) & 1u) ^ 1u,
                                                               abort_flag, true)))
                    break;
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kBN);
                for (int kb = 0; kb < p.nk; ++kb) {
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[s], ph, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        // Descriptors count in 16 bytes and do not carry out of their
                        // address field: all of shared memory is below 2^18.
                        const uint64_t w_desc = w_desc0 + (uint64_t)(s * (Shape::kStage / 16));
                        const uint64_t t_desc = w_desc + X_W_BYTES / 16;
                        const uint32_t sfw = tmem_base + (uint32_t)(Shape::kSfCol + sb * X_SF_COLS);
                        const uint32_t sft = sfw + 8;
                        tc_mma_mxf4_pair(d_tmem, w_desc, t_desc, id0, sfw, sft, kb != 0 ? 1u : 0u);
                        tc_mma_mxf4_pair(d_tmem, w_desc + 2, t_desc + 2, id2, sfw, sft, 1u);
                        tc_mma_mxf4_pair(d_tmem, w_desc + 4, t_desc + 4, id0, sfw + 4, sft + 8, 1u);
                        tc_mma_mxf4_pair(d_tmem, w_desc + 6, t_desc + 6, id2, sfw + 4, sft + 8, 1u);
                        tc_commit_pair(&empty[s], 0x3);
                        if (kb == p.nk - 1) tc_commit_pair(&tfull[acc], 0x3);
                    }
                    __syncwarp();
                    if (++s == stages) { s = 0; ph ^= 1u; }
                    if (++sb == sf_bufs) sb = 0;
                }
                tile += n_pairs;
                c.step(dt, dn, p.nt, tile < total, table);
            }
            // every MMA issued here completes before either CTA frees TMEM
            if (elect_one()) tc_commit_pair(&drain[0], 0x1);
            __syncwarp();
            wait_drained(&drain[0], abort_flag);
        }
    } else if (warp == 2) {
        if (leader) {
            // ---------------- scale copies (leader CTA) ----------------
            // A K block's scales go to the tensor memory of both CTAs as soon as
            // the last MMAs that read the buffer, sf_bufs K blocks back, have
            // completed; their completion is the second of the two arrivals that
            // the stage's MMAs wait for.
            int s = 0, sg = 0, sb = 0;
            int s2 = 0, lag = sf_bufs;  // the stage sf_bufs K blocks back
            uint32_t ph2 = 0, phg = 0;
            bool ok = true;
            const uint64_t f_desc0 = sdesc_scales(smem_u32(sfs));
            MxTile c(pair_id, p.nt, total, table);
            for (int tile = pair_id; ok && tile < total;) {
                const bool wide = c.n > 128;
                for (int kb = 0; kb < p.nk; ++kb) {
                    const int k4 = kb % X_GROUP;
                    bool got = true;
                    if (k4 == 0) got = mbar_wait_bounded(&sfull[sg], phg, abort_flag, true);
                    if (lag > 0) {
                        --lag;
                    } else {
                        got = got && mbar_wait_bounded(&empty[s2], ph2, abort_flag);
                        if (++s2 == stages) { s2 = 0; ph2 ^= 1u; }
                    }
                    if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                    tc_fence_after();
                    const bool last = k4 == X_GROUP - 1 || kb == p.nk - 1;
                    if (elect_one()) {
                        const uint64_t f_desc =
                            f_desc0 + (uint64_t)(sg * (X_GROUP_BYTES / 16) + k4 * (X_SF_BYTES / 16));
                        const uint32_t sfw = tmem_base + (uint32_t)(Shape::kSfCol + sb * X_SF_COLS);
                        const uint32_t sft = sfw + 8;
                        // blocks 0, 1: the weights' K halves; 2 + 2 half + token / 128: the tokens'
                        constexpr uint64_t kBlk = X_SF_BLOCK / 16;
                        tc_cp_scales_pair(sfw, f_desc);
                        tc_cp_scales_pair(sfw + 4, f_desc + kBlk);
                        tc_cp_scales_pair(sft, f_desc + 2 * kBlk);
                        tc_cp_scales_pair(sft + 8, f_desc + 4 * kBlk);
                        if (wide) {
                            tc_cp_scales_pair(sft + 4, f_desc + 3 * kBlk);
                            tc_cp_scales_pair(sft + 12, f_desc + 5 * kBlk);
                        }
                        tc_commit_pair(&full[s], 0x1);
                        if (last) tc_commit_pair(&sempty[sg], 0x3);
                    }
                    __syncwarp();
                    if (++s == stages) s = 0;
                    if (++sb == sf_bufs) sb = 0;
                    if (last && ++sg == X_SLOTS) { sg = 0; phg ^= 1u; }
                }
                tile += n_pairs;
                c.step(dt, dn, p.nt, tile < total, table);
            }
            if (elect_one()) tc_commit_pair(&drain[1], 0x1);
            __syncwarp();
            wait_drained(&drain[1], abort_flag);
        }
    } else if (warp >= 3 + X_SF_WARPS) {
        // ---------------- epilogue (both CTAs) ----------------
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const int ew = warp - 3 - X_SF_WARPS, eg = ew >> 2;
        const uint32_t tempty_leader = mapa_shared(smem_u32(&tempty[0]), 0);
        int it = 0;
        bool over = false;  // a stored y beyond the fp16 range
        MxTile c(pair_id, p.nt, total, table);
        for (int tile = pair_id; tile < total; ++it) {
            const int acc = it & 1;
            // the warp together (the aligned barriers and loads below need it so)
            const bool got = __all_sync(
                0xffffffffu, mbar_wait_bounded(&tfull[acc], (uint32_t)(it >> 1) & 1u, abort_flag));
            // a group's warps go on, or stop, together
            if (!bar_and(X_EPI_BAR + eg, 128, got)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kBN);
            // The accumulator is the MMA's again once every warp has its last chunk in
            // registers: tensor memory only, so the tcgen05 fences around a relaxed
            // arrival are all it takes.
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster_relaxed(tempty_leader + (uint32_t)(acc * sizeof(uint64_t)));
            };
            constexpr int kChunk = kGemm1 ? Shape::kChunk1 : 32;
            constexpr int step = kChunk * X_EPI_GROUPS;
            const bool none = kChunk * eg >= c.nvalid ||
                              (!kGemm1 && c.nt * X_BM + (int)rank * 128 + q * 32 >= p.n_out);
            if (none) release();
            if (kGemm1) {
                // lanes 0-63 are the gates of units `unit0`.., 64-127 their ups
                const int unit0 = c.nt * X_UNITS + (int)rank * 64;
                // A lane turns kUnits of a token's 64, kLanes share a block of 32 and
                // 2 kLanes a token, so that the warp stores whole 32-byte sectors of h
                // and both of a token's scales at once (16 bytes and a byte at a time: a
                // long Zipf-skewed call 844 against 834 us, others the same).  Units 32
                // on are kept with their 8s swapped in pairs (column ^ 8): the two
                // blocks' lanes would read the same banks.
                constexpr int kLanes = 64 / kChunk;
                constexpr int kUnits = 32 / kLanes;
                const int tok = q * (kChunk / 4) + lane / (2 * kLanes);  // of the chunk in the buffer
                const int blk = lane / kLanes & 1, first = lane % kLanes * kUnits;
                const int unit = blk * 32 + first;
                const bool both = (p.n_out & 63) == 0;  // a token's two scales lie on 2 bytes
                float *buf = reinterpret_cast<float *>(turn) + eg * (kChunk * X_TURN_LD);
                for (int t0 = kChunk * eg; t0 < c.nvalid; t0 += step) {
                    uint32_t d[kChunk];
                    tmem_ld_32x32b(tb + t0, d);
                    tc_wait_ld();
                    if (t0 + step >= c.nvalid) release();
                    bar_sync(X_EPI_BAR + eg, 128);  // the group has read its last chunk
#pragma unroll
                    for (int j = 0; j < kChunk; ++j)
                        buf[j * X_TURN_LD + q * 32 + (lane ^ (q & 1) << 3)] = __uint_as_float(d[j]);
                    bar_sync(X_EPI_BAR + eg, 128);
                    const float *src = buf + tok * X_TURN_LD + blk * 32;
                    float h[kUnits];
                    uint32_t top = 0;
#pragma unroll
                    for (int v = 0; v < kUnits / 4; ++v) {
                        const int at = (first + 4 * v) ^ blk << 3;
                        const float4 g = *reinterpret_cast<const float4 *>(src + at);
                        const float4 u = *reinterpret_cast<const float4 *>(src + 64 + at);
                        h[4 * v] = mx_silu(g.x) * u.x;
                        h[4 * v + 1] = mx_silu(g.y) * u.y;
                        h[4 * v + 2] = mx_silu(g.z) * u.z;
                        h[4 * v + 3] = mx_silu(g.w) * u.w;
                    }
#pragma unroll
                    for (int i = 0; i < kUnits; ++i) top = max(top, abs_bits(h[i]));
#pragma unroll
                    for (int o = 1; o < kLanes; o *= 2)  // the block's other units
                        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const uint32_t sb = mx_scale_byte(top);
                    const float inv = mx_inv_scale(sb);
                    const uint32_t sb1 = __shfl_down_sync(0xffffffffu, sb, kLanes);  // the second block's
                    if (t0 + tok < c.nvalid && unit0 + unit < p.n_out) {
                        const size_t row = (size_t)(c.row0 + t0 + tok);
                        uint32_t *to = reinterpret_cast<uint32_t *>(
                            p.hq + row * (size_t)(p.n_out / 2) + (unit0 + unit) / 2);
                        const uint32_t c0 = mx_codes8(*reinterpret_cast<const float(*)[8]>(h), inv);
                        if constexpr (kUnits == 16)
                            *reinterpret_cast<uint2 *>(to) = make_uint2(
                                c0, mx_codes8(*reinterpret_cast<const float(*)[8]>(h + 8), inv));
                        else
                            *to = c0;
                        uint8_t *sf = p.hsf + row * (size_t)(p.n_out / 32) + (unit0 + unit) / 32;
                        if (both) {
                            if (unit == 0) *reinterpret_cast<uint16_t *>(sf) = (uint16_t)(sb | sb1 << 8);
                        } else if (first == 0) {
                            *sf = (uint8_t)sb;
                        }
                    }
                }
            } else {
                // The warp's 32 columns of y, 32 tokens at a time: loaded as the
                // fragments of 8 x 8 matrices (a column of y by tokens), rounded to
                // fp16 and stored transposed, a token's 8 columns in 16 bytes; 16-byte
                // unit u of token t is kept at u ^ (t / 2 & 3), free of bank conflicts
                // both ways.  (One STS per value instead: a long Zipf-skewed call 883
                // against 849 us.)
                const int col0 = c.nt * X_BM + (int)rank * 128 + q * 32;
                uint8_t *buf = turn + ew * (32 * 64);
                const int mr = lane & 7, mf = lane >> 3;   // the address this lane gives: token, unit
                const uint32_t st = smem_u32(buf) + mr * 64 + ((mf ^ (mr >> 1 & 3)) << 4);
                if (!none) {  // (D is a multiple of 32: a warp's columns are all there or none is)
                    for (int t0 = kChunk * eg; t0 < c.nvalid; t0 += step) {
                        uint32_t d0[16], d1[16];
                        tmem_ld_16x256b_x4(tb + t0, d0);
                        tmem_ld_16x256b_x4(tb + (16u << 16) + t0, d1);
                        tc_wait_ld();
                        if (t0 + step >= c.nvalid) release();
                        // only stored values count: columns past the tile's tokens hold anything
                        if (t0 + kChunk <= c.nvalid) {
                            float top = 0.f;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(d0[i])), fabsf(__uint_as_float(d1[i]))));
                            over |= top >= kHalfOverflow;
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const bool held = t0 + 8 * (i >> 2) + 2 * (lane & 3) + (i & 1) < c.nvalid;
                                over |= held && (fabsf(__uint_as_float(d0[i])) >= kHalfOverflow ||
                                                 fabsf(__uint_as_float(d1[i])) >= kHalfOverflow);
                            }
                        }
                        __syncwarp();  // the last chunk has been read
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            auto half2 = [](const uint32_t (&d)[16], int j) {
                                return pack_half2(__uint_as_float(d[j]), __uint_as_float(d[j + 1]));
                            };
                            stmatrix_x4_trans(st + i * (8 * 64), half2(d0, 4 * i), half2(d0, 4 * i + 2),
                                              half2(d1, 4 * i), half2(d1, 4 * i + 2));
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int tok = 8 * i + (lane >> 2);
                            if (t0 + tok < c.nvalid)
                                *reinterpret_cast<uint4 *>(
                                    p.y + (size_t)(c.row0 + t0 + tok) * p.n_out + col0 + (lane & 3) * 8) =
                                    *reinterpret_cast<const uint4 *>(
                                        buf + tok * 64 + (((lane & 3) ^ (tok >> 1 & 3)) << 4));
                        }
                    }
                }
            }
            tile += n_pairs;
            c.step(dt, dn, p.nt, tile < total, table);
        }
        if (!kGemm1 && __any_sync(0xffffffffu, over) && lane == 0) raise_flag(p.status, FLAG_RANGE);
    } else {
        // ---------------- scale fetchers (both CTAs) ----------------
        const int w = warp - 3, slot = w >> 1;
        const ScaleWarp f{sfs + slot * X_GROUP_BYTES, &sempty[slot],
                          mapa_shared(smem_u32(&sfull[slot]), 0), abort_flag, slot, lane,
                          pair_id, n_pairs, dt, dn, (int)rank};
        if ((p.K / 32 & 3) == 0) {
            if (w & 1)
                fetch_scales<kGemm1, true, kBN, true>(f, p, table);
            else
                fetch_scales<kGemm1, false, kBN, true>(f, p, table);
        } else {
            if (w & 1)
                fetch_scales<kGemm1, true, kBN, false>(f, p, table);
            else
                fetch_scales<kGemm1, false, kBN, false>(f, p, table);
        }
    }

    tc_fence_before();
    __syncthreads();
    // after an abort loads may be in flight for stages the MMA warp never
    // consumed; the peer waits at the cluster barrier too
    if (threadIdx.x == 0 && *abort_flag) settle_inflight_copies();
    cluster_sync();  // the leader's MMAs (which read both CTAs' smem) are done
    if (threadIdx.x == 0 && *abort_flag) {
        raise_flag(p.status, FLAG_TIMEOUT);
        atomicCAS(p.status + 1, 0, 1 + blockIdx.x);
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, X_TMEM_COLS);
    }
}

// Clusters of two that fit at once on the current device (0 if none), asked once
// for the largest launch: one CTA takes an SM whatever the number of experts, by its
// ring in shared memory as by its 512 columns of tensor memory.
template <bool kGemm1, int kBN>
int max_mx_clusters() {
    constexpr int kMaxDev = 64;
    static std::atomic<int> cached[kMaxDev];  // threads launch at once
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
    if (const int n = cached[dev].load(std::memory_order_relaxed)) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 256);
    cfg.blockDim = dim3(X_THREADS);
    cfg.dynamicSmemBytes = X_SMEM_MAX;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (void *)grouped_mx_kernel<kGemm1, kBN>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

struct MxMaps {
    CUtensorMap t8, t16, t32, t64, w0, w1;
};

// Token boxes of 8, 16, 32 and 64 rows; a tile of at most 32 tokens loads 8 or
// 16 per CTA, and the others only have to be valid.
bool token_maps(MxMaps *m, const uint8_t *codes, int K, int64_t rows, int bn) {
    if (!make_tmap_tile(&m->t8, codes, 1, K / 2, rows, 0, X_ROW, 8, 128) ||
        !make_tmap_tile(&m->t16, codes, 1, K / 2, rows, 0, X_ROW, 16, 128))
        return false;
    m->t32 = m->t64 = m->t16;
    return bn <= 32 || (make_tmap_tile(&m->t32, codes, 1, K / 2, rows, 0, X_ROW, 32, 128) &&
                        make_tmap_tile(&m->t64, codes, 1, K / 2, rows, 0, X_ROW, 64, 128));
}

template <bool kGemm1, int kBN>
cudaError_t launch_mx(const MxMaps &m, MxParams p, long long token_tiles, cudaStream_t stream) {
    static_assert(1024 + 4 * MxShape<kBN>::kStage + X_SLOTS * X_GROUP_BYTES + MxShape<kBN>::kTurn1 +
                          (X_NBARS + 1) * 8 + 16 + 4 * (4 * 1024 + 1) <= X_SMEM_MAX,
                  "four stages fit beside the table of 1024 experts");
    int stages = X_MAX_STAGES;  // as many as fit beside the table of the experts
    while (mx_smem_bytes<kGemm1, kBN>(stages, p.E_local) > X_SMEM_MAX) --stages;
    p.stages = stages;
    const size_t smem = mx_smem_bytes<kGemm1, kBN>(stages, p.E_local);
    cudaError_t e = ensure_smem((const void *)grouped_mx_kernel<kGemm1, kBN>, X_SMEM_MAX);
    if (e != cudaSuccess) return e;
    const int clusters = max_mx_clusters<kGemm1, kBN>();
    if (clusters <= 0) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)std::min<long long>(clusters, token_tiles * p.nt));
    cfg.blockDim = dim3(X_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = MOE_PDL ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, grouped_mx_kernel<kGemm1, kBN>, m.t8, m.t16, m.t32, m.t64, m.w0, m.w1, p);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <int kBN>
cudaError_t launch_mx_both(const MxMaps &m1, const MxMaps &m2, const MxParams &p1, const MxParams &p2,
                           cudaStream_t stream) {
    // token tiles: at most one partial tile per expert beside the whole ones
    const long long tt = std::min<long long>(p1.rows_alloc, p1.rows_alloc / kBN + p1.E_local);
    const cudaError_t e = launch_mx<true, kBN>(m1, p1, tt, stream);
    return e == cudaSuccess ? launch_mx<false, kBN>(m2, p2, tt, stream) : e;
}

}  // namespace

cudaError_t launch_grouped_swiglu_mxfp4(const uint8_t *x_perm_q, const uint8_t *x_scale,
                                        const int *seg_offsets, const int *tokens_per_expert,
                                        const MxWeights &w, uint8_t *h_q, uint8_t *h_scale,
                                        void *y_perm, int D, int H_local, int e_first, int E_local,
                                        int64_t rows_alloc, double avg_rows, int *status,
                                        cudaStream_t stream) {
    if (E_local == 0 || rows_alloc == 0) return cudaSuccess;
    if (D % 32 || H_local % 32) return cudaErrorInvalidValue;
    MxParams p{};
    p.E_local = E_local;
    p.e_first = e_first;
    p.rows_alloc = (int)rows_alloc;
    p.seg_off = seg_offsets;
    p.tpe = tokens_per_expert;
    p.status = status;

    MxParams p1 = p;
    p1.K = D;
    p1.nk = (D + X_BK - 1) / X_BK;
    p1.n_out = H_local;
    p1.nt = (H_local + X_UNITS - 1) / X_UNITS;
    p1.t_sf = x_scale;
    p1.w_sf0 = w.w1_scale;
    p1.w_sf1 = w.w3_scale;
    p1.hq = h_q;
    p1.hsf = h_scale;

    MxParams p2 = p;
    p2.K = H_local;
    p2.nk = (H_local + X_BK - 1) / X_BK;
    p2.n_out = D;
    p2.nt = (D + X_BM - 1) / X_BM;
    p2.t_sf = h_scale;
    p2.w_sf0 = p2.w_sf1 = w.w2_scale;
    p2.y = static_cast<__half *>(y_perm);

    // Tokens per tile: 208 is the most that two accumulators leave room for; a
    // smaller tile needs less of the ring per stage and so has more stages, which
    // is worth it where it costs no further tile: the smallest of 32, 144 and 208
    // that takes an average expert's rows (and a standard deviation more) in as
    // few tiles as 208.  Grouped call on GB300, by tile: a decode batch (4 rows
    // per expert) 855 us with 32, 874 with 208; 8192 tokens over 256 experts (256
    // rows) 1282 us with 144, 1331 with 208; fine-grained (384 rows) 138 us with
    // 144, 113 with 208.
    const double rows = avg_rows + sqrt((double)avg_rows);
    auto tiles = [&](int bn) { return std::max(1LL, (long long)std::ceil(rows / bn)); };
    const int bn = tiles(32) == tiles(208) ? 32 : tiles(144) == tiles(208) ? 144 : 208;

    MxMaps m1, m2;
    if (!token_maps(&m1, x_perm_q, D, rows_alloc, bn) ||
        !token_maps(&m2, h_q, H_local, rows_alloc, bn) ||
        !make_tmap_tile(&m1.w0, w.w1, 1, D / 2, H_local, E_local, X_ROW, 64, 128) ||
        !make_tmap_tile(&m1.w1, w.w3, 1, D / 2, H_local, E_local, X_ROW, 64, 128) ||
        !make_tmap_tile(&m2.w0, w.w2, 1, H_local / 2, D, E_local, X_ROW, 128, 128))
        return cudaErrorInvalidValue;
    m2.w1 = m2.w0;
    return bn == 32    ? launch_mx_both<32>(m1, m2, p1, p2, stream)
           : bn == 144 ? launch_mx_both<144>(m1, m2, p1, p2, stream)
                       : launch_mx_both<208>(m1, m2, p1, p2, stream);
}

}  // namespace moe
