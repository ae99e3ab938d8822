// MXFP4 m-grouped SwiGLU expert FFN (tcgen05 kind::mxf4, block scales).
//
// Same contract as grouped_tc.cu over operands of e2m1 codes with one e8m0
// scale per 32 elements of K (mxfp4_row.cuh):
//   g = sum_b 2^(ex[r,b] + e1[n,b]) sum_{i in b} qx[r,i] q1[n,i],  u with w3,
//   h = mxfp4(SiLU(g) u),  y = fp16(h w2^T).
// Products of codes are exact, the tensor cores apply the scales and sum in
// fp32; h is rounded once, from the fp32 result straight to MXFP4 (GEMM2's
// operand), and y once to fp16, as the other bf16 layers store it.
//
// Each GEMM is one persistent launch of one CTA per SM over 128 x 192 output
// tiles, K in blocks of 256 elements (128 packed bytes, a 128-byte swizzled
// row):
//   * GEMM1's 192 columns are the gate and the up products of the same 96
//     hidden units, so the epilogue has both in one lane; a lane holds one
//     row, so a block of 32 hidden units is 32 registers of one thread and
//     its maximum needs no exchange;
//   * N = 192 leaves 128 of the 512 tensor-memory columns beside two
//     accumulators: the scales of five K blocks (24 columns each), one buffer
//     per pipeline stage, so scales are never overwritten under an MMA;
//   * scales are read in their natural [rows, K / 32] layout, which is not the
//     order the tensor cores want (four scales each of rows l, l + 32, l + 64
//     and l + 96 together): four warps gather them, one per stage in flight,
//     into 512-byte blocks that tcgen05.cp spreads over tensor memory;
//   * a tile of at most 64 valid rows loads only those (16-row boxes); the
//     other rows of the operand are whatever the stage held -- every code is a
//     finite number and their scales are set to 1 -- and are not stored;
//   * every mbarrier wait is bounded (FLAG_TIMEOUT).
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "mxfp4_row.cuh"

namespace moe {
namespace {

constexpr int X_BM = 128;             // token rows per tile
constexpr int X_BN = 192;             // output columns per tile (GEMM1: 96 gate, 96 up)
constexpr int X_UNITS = X_BN / 2;     // hidden units per GEMM1 tile
constexpr int X_BK = 256;             // K elements per stage
constexpr int X_ROW = X_BK / 2;       // bytes of a row's K block: the swizzle span
constexpr int X_A_BYTES = X_BM * X_ROW;
constexpr int X_B_BYTES = X_BN * X_ROW;
constexpr int X_SF_BLOCK = 512;       // 128 rows x 4 scales
constexpr int X_SF_BYTES = 6 * X_SF_BLOCK;  // two K halves of A's block, then of B's two
constexpr int X_STAGE_BYTES = X_A_BYTES + X_B_BYTES + X_SF_BYTES;
constexpr int X_MAX_STAGES = 5;
constexpr int X_EPI_WARPS = 4;
constexpr int X_SF_WARPS = 4;
constexpr int X_THREADS = 64 + 32 * (X_EPI_WARPS + X_SF_WARPS);
constexpr int X_TMEM_COLS = 512;
constexpr int X_SF_COL = 2 * X_BN;    // scale buffers start here
constexpr int X_SF_COLS = 24;         // per stage: 2 x 4 for A, 2 x 8 for B
static_assert(X_SF_COL + X_MAX_STAGES * X_SF_COLS <= X_TMEM_COLS, "tensor memory columns");
static_assert(X_STAGE_BYTES % 1024 == 0, "stages keep the swizzle's alignment");
constexpr int X_NBARS = 2 * X_MAX_STAGES + 5;
constexpr int X_SMEM_MAX = 227 * 1024;

struct MxParams {
    int E_local, e_first, rows_alloc;
    int stages;
    int K, nk;            // reduction length (D or H_local) and its 256-blocks
    int nt, n_out;        // tiles along N; columns of the output (H_local or D)
    const int *seg_off, *tpe;
    const uint8_t *a_sf;          // [rows_alloc, K / 32]
    const uint8_t *b_sf0, *b_sf1; // w1 and w3 [E_local, H_local, D / 32], or w2 twice
    uint8_t *hq, *hsf;            // GEMM1: codes [rows, H / 2], scales [rows, H / 32]
    __half *y;                    // GEMM2: [rows, D]
    int *status;
};

size_t mx_smem_bytes(int stages, int E_local) {
    return 1024 + (size_t)stages * X_STAGE_BYTES + (X_NBARS + 1) * sizeof(uint64_t) + 16 +
           sizeof(int) * (3 * (size_t)E_local + 1);
}

struct MxTile {
    int expert, row0, nvalid, nt;
};

__device__ __forceinline__ MxTile decode_tile(int v, const MxParams &p, const int *s_mtoff,
                                              const int *s_base, const int *s_valid) {
    MxTile c;
    const int mt = v / p.nt;
    c.nt = v - mt * p.nt;
    c.expert = tile_expert(s_mtoff, p.E_local, mt);
    const int lm = mt - s_mtoff[c.expert];
    c.row0 = s_base[c.expert] + lm * X_BM;
    c.nvalid = min(X_BM, s_valid[c.expert] - lm * X_BM);
    return c;
}

// SiLU(g) = g / (1 + e^-g) with the fast approximate division (2 ulp in fp32,
// far below the 4-bit rounding); 0 where e^-g overflows, as SiLU is there.
__device__ __forceinline__ float mx_silu(float g) { return __fdividef(g, 1.f + __expf(-g)); }

// The 8 scales of a row's K block kb: bytes [8 kb, 8 kb + 8) of its `ld`
// scales, 1.0 (byte 127) past the end (the codes there are zeros).
__device__ __forceinline__ uint2 load_scales(const uint8_t *row, int kb, int ld) {
    const int b = kb * 8;
    uint2 v = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    if ((ld & 7) == 0) {
        v = *reinterpret_cast<const uint2 *>(row + b);
    } else if ((ld & 3) == 0) {
        v.x = *reinterpret_cast<const uint32_t *>(row + b);
        if (b + 4 < ld) v.y = *reinterpret_cast<const uint32_t *>(row + b + 4);
    } else {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i >> 2] |= (b + i < ld ? (uint32_t)row[b + i] : 127u) << (8 * (i & 3));
        v = make_uint2(w[0], w[1]);
    }
    return v;
}

template <bool kGemm1>
__global__ void __launch_bounds__(X_THREADS, 1)
grouped_mx_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA16,
                  const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                  const MxParams p) {
    griddep_launch_dependents();  // the next kernel may be scheduled now
    griddep_wait();               // every input of this kernel is complete
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + p.stages * X_STAGE_BYTES);
    uint64_t *full = bars;                       // TMA bytes + the stage's scale warp -> MMA
    uint64_t *empty = bars + X_MAX_STAGES;       // MMA -> TMA and scale warps
    uint64_t *tfull = bars + 2 * X_MAX_STAGES;   // [2] MMA -> epilogue
    uint64_t *tempty = tfull + 2;                // [2] epilogue -> MMA
    uint64_t *drain = tempty + 2;                // MMA completion at exit
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + X_NBARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *s_base = reinterpret_cast<int *>(tmem_slot + 4);
    int *s_valid = s_base + p.E_local;
    int *s_mtoff = s_valid + p.E_local;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = p.stages;
    if (warp == 0) {
        build_tile_table(lane, p.E_local, p.e_first, p.rows_alloc, X_BM, p.seg_off, p.tpe, s_base,
                         s_valid, s_mtoff, blockIdx.x == 0 ? p.status : nullptr);
        if (lane == 0) {
            for (int s = 0; s < stages; ++s) {
                mbar_init(&full[s], 2);
                mbar_init(&empty[s], 1);
            }
            for (int a = 0; a < 2; ++a) {
                mbar_init(&tfull[a], 1);
                mbar_init(&tempty[a], X_EPI_WARPS);
            }
            mbar_init(drain, 1);
            *abort_flag = 0;
            fence_mbarrier_init();
            prefetch_tmap(&tmA);
            prefetch_tmap(&tmA16);
            prefetch_tmap(&tmB0);
            if (kGemm1) prefetch_tmap(&tmB1);
        }
    } else if (warp == 1) {
        tmem_alloc(tmem_slot, X_TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total = s_mtoff[p.E_local] * p.nt;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer ----------------
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
                const MxTile c = decode_tile(tile, p, s_mtoff, s_base, s_valid);
                const int n16 = c.nvalid <= 64 ? (c.nvalid + 15) / 16 : 0;  // 16-row boxes of A
                const uint32_t tx = (n16 ? n16 * 16 * X_ROW : X_A_BYTES) + X_B_BYTES;
                for (int kb = 0; kb < p.nk; ++kb) {
                    if (!mbar_wait_bounded(&empty[s], ph ^ 1u, abort_flag)) { ok = false; break; }
                    mbar_arrive_expect_tx(&full[s], tx);
                    uint8_t *sa = ring + s * X_STAGE_BYTES;
                    uint8_t *sb = sa + X_A_BYTES;
                    if (n16)
                        for (int i = 0; i < n16; ++i)
                            tma_load_2d(sa + i * 16 * X_ROW, &tmA16, &full[s], kb * X_ROW,
                                        c.row0 + 16 * i);
                    else
                        tma_load_2d(sa, &tmA, &full[s], kb * X_ROW, c.row0);
                    if (kGemm1) {
                        tma_load_3d(sb, &tmB0, &full[s], kb * X_ROW, c.nt * X_UNITS, c.expert);
                        tma_load_3d(sb + X_B_BYTES / 2, &tmB1, &full[s], kb * X_ROW,
                                    c.nt * X_UNITS, c.expert);
                    } else {
                        tma_load_3d(sb, &tmB0, &full[s], kb * X_ROW, c.nt * X_BN, c.expert);
                    }
                    if (++s == stages) { s = 0; ph ^= 1u; }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            int it = 0;
            for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x, ++it) {
                const int acc = it & 1;
                if (!mbar_wait_bounded(&tempty[acc], ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag))
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * X_BN);
                for (int kb = 0; kb < p.nk; ++kb) {
                    if (!mbar_wait_bounded(&full[s], ph, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(ring + s * X_STAGE_BYTES);
                    const uint32_t b_addr = a_addr + X_A_BYTES;
                    const uint32_t f_addr = b_addr + X_B_BYTES;
                    const uint32_t sfa = tmem_base + (uint32_t)(X_SF_COL + s * X_SF_COLS);
                    const uint32_t sfb = sfa + 8;
                    // blocks 0, 1: A's K halves; 2 + 2 half + rows / 128: B's.  The
                    // copies and the MMAs of one thread execute in issue order.
#pragma unroll
                    for (int b = 0; b < 6; ++b)
                        tc_cp_scales(sfa + 4 * b, sdesc_scales(f_addr + b * X_SF_BLOCK));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_mxf4(d_tmem, sdesc_kmajor_sw128(a_addr + kk * 32),
                                    sdesc_kmajor_sw128(b_addr + kk * 32),
                                    idesc_mxf4_f32(X_BM, X_BN, 2 * (kk & 1)), sfa + 4 * (kk >> 1),
                                    sfb + 8 * (kk >> 1), (kb | kk) != 0 ? 1u : 0u);
                    tc_commit(&empty[s]);
                    if (++s == stages) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                tc_commit(&tfull[acc]);
            }
            // every MMA issued here completes before TMEM is freed
            tc_commit(drain);
            volatile int local_abort = 0;
            mbar_wait_bounded(drain, 0u, &local_abort);
        }
    } else if (warp < 2 + X_EPI_WARPS) {
        // ---------------- epilogue (warps 2..5) ----------------
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const int r = q * 32 + lane;
        int it = 0;
        for (int tile = blockIdx.x; tile < total; tile += gridDim.x, ++it) {
            const MxTile c = decode_tile(tile, p, s_mtoff, s_base, s_valid);
            const int acc = it & 1;
            const bool got = mbar_wait_bounded(&tfull[acc], (uint32_t)(it >> 1) & 1u, abort_flag);
            if (!__all_sync(0xffffffffu, got)) break;
            tc_fence_after();
            const bool row_ok = r < c.nvalid;
            const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * X_BN);
            if (q * 32 < c.nvalid) {
                if (kGemm1) {
                    const size_t row = (size_t)(c.row0 + (row_ok ? r : 0));
#pragma unroll 1
                    for (int b = 0; b < X_UNITS / 32; ++b) {
                        const int unit = c.nt * X_UNITS + b * 32;
                        if (unit >= p.n_out) break;  // uniform: H_local is a multiple of 32
                        uint32_t g[32], u[32];
                        tmem_ld_32x32b_x32(tb + b * 32, g);
                        tmem_ld_32x32b_x32(tb + X_UNITS + b * 32, u);
                        tc_wait_ld();
                        float h[32];
                        uint32_t top = 0;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            h[i] = mx_silu(__uint_as_float(g[i])) * __uint_as_float(u[i]);
                            top = max(top, abs_bits(h[i]));
                        }
                        const uint32_t sb = mx_scale_byte(top);
                        const float inv = mx_inv_scale(sb);
                        uint32_t w[4];
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            w[v] = mx_codes8(*reinterpret_cast<const float(*)[8]>(h + 8 * v), inv);
                        if (row_ok) {
                            *reinterpret_cast<uint4 *>(p.hq + row * (size_t)(p.n_out / 2) + unit / 2) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                            p.hsf[row * (size_t)(p.n_out / 32) + unit / 32] = (uint8_t)sb;
                        }
                    }
                } else {
                    __half *yrow = p.y + (size_t)(c.row0 + (row_ok ? r : 0)) * p.n_out;
                    bool over = false;  // a stored value beyond the fp16 range
#pragma unroll 1
                    for (int b = 0; b < X_BN / 32; ++b) {
                        const int col0 = c.nt * X_BN + b * 32;
                        if (col0 >= p.n_out) break;  // uniform: D is a multiple of 32
                        uint32_t d[32];
                        tmem_ld_32x32b_x32(tb + b * 32, d);
                        tc_wait_ld();
                        if (!row_ok) continue;
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float lo = __uint_as_float(d[v * 8 + 2 * i]);
                                const float hi = __uint_as_float(d[v * 8 + 2 * i + 1]);
                                over |= fabsf(lo) >= kHalfOverflow || fabsf(hi) >= kHalfOverflow;
                                w[i] = pack_half2(lo, hi);
                            }
                            *reinterpret_cast<uint4 *>(yrow + col0 + v * 8) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    if (__any_sync(0xffffffffu, over) && lane == 0) raise_flag(p.status, FLAG_RANGE);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[acc]);
        }
    } else {
        // ---------------- scales (warps 6..9) ----------------
        // Warp g fills the stages n with n % 4 == g.  Lane l fetches the 8
        // scales of the stage's K block for operand rows l, l + 32, ... (in
        // flight while the stage is still busy) and stores, for each K half of
        // 128 and each 128 rows, the 16 bytes of rows l, +32, +64, +96.
        const int gw = warp - 2 - X_EPI_WARPS;
        const int ld = p.K / 32;
        int s = 0;
        uint32_t ph = 0, n = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
            const MxTile c = decode_tile(tile, p, s_mtoff, s_base, s_valid);
            for (int kb = 0; kb < p.nk; ++kb, ++n) {
                if ((int)(n % X_SF_WARPS) == gw) {
                    uint2 a[4], b[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i] = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
                        if (lane + 32 * i < c.nvalid)
                            a[i] = load_scales(p.a_sf + (size_t)(c.row0 + lane + 32 * i) * ld, kb, ld);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        b[i] = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
                        if (i >= X_BN / 32) continue;
                        // operand row lane + 32 i: a gate or an up row, or a row of w2
                        const bool up = kGemm1 && i >= X_UNITS / 32;
                        const int wr = kGemm1 ? c.nt * X_UNITS + lane + 32 * (up ? i - X_UNITS / 32 : i)
                                              : c.nt * X_BN + lane + 32 * i;
                        if (wr < p.n_out)
                            b[i] = load_scales((up ? p.b_sf1 : p.b_sf0) +
                                                   ((size_t)c.expert * p.n_out + wr) * ld, kb, ld);
                    }
                    bool got = true;
                    if (lane == 0) got = mbar_wait_bounded(&empty[s], ph ^ 1u, abort_flag);
                    if (!__shfl_sync(0xffffffffu, got, 0)) { ok = false; break; }
                    uint4 *f = reinterpret_cast<uint4 *>(ring + s * X_STAGE_BYTES + X_A_BYTES + X_B_BYTES) + lane;
                    f[0] = make_uint4(a[0].x, a[1].x, a[2].x, a[3].x);
                    f[32] = make_uint4(a[0].y, a[1].y, a[2].y, a[3].y);
                    f[64] = make_uint4(b[0].x, b[1].x, b[2].x, b[3].x);
                    f[96] = make_uint4(b[4].x, b[5].x, b[6].x, b[7].x);
                    f[128] = make_uint4(b[0].y, b[1].y, b[2].y, b[3].y);
                    f[160] = make_uint4(b[4].y, b[5].y, b[6].y, b[7].y);
                    fence_proxy_async_smem();  // tcgen05.cp reads them through the async proxy
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[s]);
                }
                if (++s == stages) { s = 0; ph ^= 1u; }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        // loads may be in flight for stages the MMA warp never consumed
        settle_inflight_copies();
        raise_flag(p.status, FLAG_TIMEOUT);
        atomicCAS(p.status + 1, 0, 1 + blockIdx.x);
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, X_TMEM_COLS);
    }
}

}  // namespace

cudaError_t launch_grouped_swiglu_mxfp4(const uint8_t *x_perm_q, const uint8_t *x_scale,
                                        const int *seg_offsets, const int *tokens_per_expert,
                                        const MxWeights &w, uint8_t *h_q, uint8_t *h_scale,
                                        void *y_perm, int D, int H_local, int e_first, int E_local,
                                        int64_t rows_alloc, int *status, cudaStream_t stream) {
    if (E_local == 0 || rows_alloc == 0) return cudaSuccess;
    if (D % 32 || H_local % 32) return cudaErrorInvalidValue;
    // five stages leave room for the table of about 850 experts, four for any
    int stages = X_MAX_STAGES;
    while (stages > 1 && mx_smem_bytes(stages, E_local) > X_SMEM_MAX) --stages;
    const size_t smem = mx_smem_bytes(stages, E_local);
    cudaError_t e = ensure_smem((const void *)grouped_mx_kernel<true>, smem);
    if (e == cudaSuccess) e = ensure_smem((const void *)grouped_mx_kernel<false>, smem);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;

    CUtensorMap x, x16, b0, b1, h, h16, b2;
    if (!make_tmap_tile(&x, x_perm_q, 1, D / 2, rows_alloc, 0, X_ROW, X_BM, 128) ||
        !make_tmap_tile(&x16, x_perm_q, 1, D / 2, rows_alloc, 0, X_ROW, 16, 128) ||
        !make_tmap_tile(&b0, w.w1, 1, D / 2, H_local, E_local, X_ROW, X_UNITS, 128) ||
        !make_tmap_tile(&b1, w.w3, 1, D / 2, H_local, E_local, X_ROW, X_UNITS, 128) ||
        !make_tmap_tile(&h, h_q, 1, H_local / 2, rows_alloc, 0, X_ROW, X_BM, 128) ||
        !make_tmap_tile(&h16, h_q, 1, H_local / 2, rows_alloc, 0, X_ROW, 16, 128) ||
        !make_tmap_tile(&b2, w.w2, 1, H_local / 2, D, E_local, X_ROW, X_BN, 128))
        return cudaErrorInvalidValue;

    // m-tiles: at most one partial tile per expert beside the whole ones
    const long long mt = std::min<long long>(rows_alloc, rows_alloc / X_BM + E_local);
    MxParams p{};
    p.E_local = E_local;
    p.e_first = e_first;
    p.rows_alloc = (int)rows_alloc;
    p.stages = stages;
    p.seg_off = seg_offsets;
    p.tpe = tokens_per_expert;
    p.status = status;

    MxParams p1 = p;
    p1.K = D;
    p1.nk = (D + X_BK - 1) / X_BK;
    p1.n_out = H_local;
    p1.nt = (H_local + X_UNITS - 1) / X_UNITS;
    p1.a_sf = x_scale;
    p1.b_sf0 = w.w1_scale;
    p1.b_sf1 = w.w3_scale;
    p1.hq = h_q;
    p1.hsf = h_scale;
    e = launch_pdl(grouped_mx_kernel<true>, dim3((unsigned)std::min<long long>(sms, mt * p1.nt)),
                   dim3(X_THREADS), smem, stream, x, x16, b0, b1, p1);
    if (e != cudaSuccess) return e;
    count_launch();

    MxParams p2 = p;
    p2.K = H_local;
    p2.nk = (H_local + X_BK - 1) / X_BK;
    p2.n_out = D;
    p2.nt = (D + X_BN - 1) / X_BN;
    p2.a_sf = h_scale;
    p2.b_sf0 = p2.b_sf1 = w.w2_scale;
    p2.y = static_cast<__half *>(y_perm);
    e = launch_pdl(grouped_mx_kernel<false>, dim3((unsigned)std::min<long long>(sms, mt * p2.nt)),
                   dim3(X_THREADS), smem, stream, h, h16, b2, b2, p2);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace moe
