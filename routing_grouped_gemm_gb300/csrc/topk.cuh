// Top-k selection and routing weights by one warp, shared by the router's
// kernels and the layer for a few tokens.
#pragma once

#include "common.cuh"

namespace moe {

// Top-k of one token's E keys (in shared or global memory) by one warp: k rounds of a
// warp-wide arg-max in selection order (larger key first, equal keys by
// lower expert index, NaN after every number, -0 equal to +0), then the
// routing weights: softmax over all E (or sigmoid) of the chosen keys,
// divided by their sum when renormalising.  Lane i owns experts i, i+32, ...
// (E <= 1024); the winner of round j is kept by lane j, which computes and
// writes slot j.
//
// Group-limited routing (n_group > 1; page "Expert Parallelism (EP)",
// section 3): first each of the n_group groups of E/n_group consecutive
// experts is scored by the fp32 sum of its m = k/topk_group largest keys
// (added in selection order), the topk_group best groups are kept (ties to
// the lower group, NaN last), and the k rounds only consider their experts.

// The selection order as one unsigned 64-bit number, larger = chosen first.
// High word: the key's binary32 bits mapped order-preservingly onto unsigned
// integers (negative values bit-inverted, the sign bit set on the others),
// with -0 folded onto +0 and NaN mapped to 0, below every number.  Low word:
// ~e, so that of two equal keys the lower expert index is larger.  0 means
// "no candidate": a real candidate's low word ~e is nonzero.
__device__ __forceinline__ uint64_t sel_key(float v, int e) {
    uint32_t b = __float_as_uint(v);
    b = b == 0x80000000u ? 0u : b;
    uint32_t u = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    u = v != v ? 0u : u;
    return ((uint64_t)u << 32) | (uint64_t)(~(uint32_t)e);
}

// Warp-wide maximum of the lanes' selection keys (two redux.sync steps: the
// high words, then the low words of the lanes that hold the largest high
// word); every lane gets the result.
__device__ __forceinline__ uint64_t warp_max_key(uint64_t x) {
    const uint32_t hi = (uint32_t)(x >> 32);
    const uint32_t mhi = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t mlo = __reduce_max_sync(0xffffffffu, hi == mhi ? (uint32_t)x : 0u);
    return ((uint64_t)mhi << 32) | mlo;
}

__device__ __forceinline__ int key_expert(uint64_t x) { return x ? (int)~(uint32_t)x : -1; }

// KC: selection keys cached in registers per lane (E <= 32 KC); the keys are
// formed once, and each round is a masked maximum over the cache plus the
// warp-wide maximum.
template <int KC>
__device__ __forceinline__ void warp_topk_cached(const float *l, int E, int k, int score,
                                                 int renorm, int n_group, int topk_group, int t,
                                                 int *__restrict__ topk_idx,
                                                 float *__restrict__ topk_w, int *status,
                                                 int lane) {
    uint64_t key[KC];  // key[q]: expert lane + 32 q, 0 when absent
    bool any_nan = false;
#pragma unroll
    for (int q = 0; q < KC; ++q) {
        const int e = lane + 32 * q;
        const float v = e < E ? l[e] : 0.f;
        any_nan |= v != v;
        key[q] = e < E ? sel_key(v, e) : 0ull;
    }
    if (__any_sync(0xffffffffu, any_nan) && lane == 0) raise_flag(status, FLAG_BAD_ROUTING);

    const bool grouped = n_group > 1;
    uint32_t avail = 0xffffffffu;  // bit q: expert lane + 32 q may still be chosen
    if (grouped) {
        const int gsz = E / n_group;
        const int m = k / topk_group;
        float my_score = 0.f;  // lane g: score of group g
        for (int g = 0; g < n_group; ++g) {
            const int e0 = g * gsz;
            uint32_t in = 0;  // bit q: expert lane + 32 q is in group g
#pragma unroll
            for (int q = 0; q < KC; ++q) {
                const int e = lane + 32 * q;
                if (e >= e0 && e < e0 + gsz) in |= 1u << q;
            }
            float sum = 0.f;
            for (int i = 0; i < m; ++i) {
                uint64_t best = 0;
#pragma unroll
                for (int q = 0; q < KC; ++q) {
                    const uint64_t c = ((in >> q) & 1u) ? key[q] : 0ull;
                    best = c > best ? c : best;
                }
                const int be = key_expert(warp_max_key(best));
                if (be >= 0 && (be & 31) == lane) in &= ~(1u << (be >> 5));
                sum += be >= 0 ? l[be] : 0.f;
            }
            if (lane == g) my_score = sum;
        }
        uint32_t allowed = 0;  // bit g: group g may be chosen
        for (int r = 0; r < topk_group; ++r) {
            const uint64_t c =
                (lane < n_group && !(allowed & (1u << lane))) ? sel_key(my_score, lane) : 0ull;
            const int bg = key_expert(warp_max_key(c));
            if (bg >= 0) allowed |= 1u << bg;
        }
        avail = 0;
#pragma unroll
        for (int q = 0; q < KC; ++q) {
            const int e = lane + 32 * q;
            if (e < E && ((allowed >> (e / gsz)) & 1u)) avail |= 1u << q;
        }
    }

    int my_e = -1;  // slot `lane`'s expert and key (lanes < k)
    float my_v = 0.f, top = 0.f;
    for (int j = 0; j < k; ++j) {
        uint64_t best = 0;
#pragma unroll
        for (int q = 0; q < KC; ++q) {
            const uint64_t c = ((avail >> q) & 1u) ? key[q] : 0ull;
            best = c > best ? c : best;
        }
        const int be = key_expert(warp_max_key(best));
        const float bv = be >= 0 ? l[be] : 0.f;
        if (be >= 0 && (be & 31) == lane) avail &= ~(1u << (be >> 5));
        if (lane == j) { my_e = be; my_v = bv; }
        if (j == 0) top = bv;  // the largest chosen key (unless NaN)
    }
    if (grouped && score == 0 && !renorm) {
        // softmax over all E: shift by the largest key of all, which may lie
        // in a group that was not chosen
        uint64_t best = 0;
#pragma unroll
        for (int q = 0; q < KC; ++q) best = key[q] > best ? key[q] : best;
        const int be = key_expert(warp_max_key(best));
        top = be >= 0 ? l[be] : 0.f;
    }

    float p = 0.f;
    if (lane < k) p = (score == 0) ? expf(my_v - top) : 1.f / (1.f + expf(-my_v));
    float div = 1.f;
    if (renorm) {
        float sum = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        div = sum;
    } else if (score == 0) {
        float sum = 0.f;
        for (int e = lane; e < E; e += 32) sum += expf(l[e] - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        div = sum;
    }
    if (lane < k) {
        topk_idx[(size_t)t * k + lane] = my_e;
        topk_w[(size_t)t * k + lane] = p / div;
    }
}

// EMAX: the largest E the calling kernel handles (256 or 1024).
template <int EMAX>
__device__ void warp_topk_weights(const float *l, int E, int k, int score, int renorm,
                                  int n_group, int topk_group, int t,
                                  int *__restrict__ topk_idx, float *__restrict__ topk_w,
                                  int *status, int lane) {
    if (E <= 64)
        warp_topk_cached<2>(l, E, k, score, renorm, n_group, topk_group, t, topk_idx, topk_w,
                            status, lane);
    else if (EMAX <= 256 || E <= 256)
        warp_topk_cached<8>(l, E, k, score, renorm, n_group, topk_group, t, topk_idx, topk_w,
                            status, lane);
    else
        warp_topk_cached<32>(l, E, k, score, renorm, n_group, topk_group, t, topk_idx, topk_w,
                             status, lane);
}

}  // namespace moe
