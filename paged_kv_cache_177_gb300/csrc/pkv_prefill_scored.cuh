// pkv_prefill_scored.cuh -- prefill attention with transformed scores on the
// 5th-generation tensor cores: scores capped by a tanh, biased by distance, cut
// to a window, over a prefix that is seen from both sides.
#pragma once

#include <algorithm>
#include <cfloat>
#include <cmath>

#include <cooperative_groups.h>

#include "pkv_prefill_tc.cuh"

namespace pkv {

struct ScoredPrefillParams {
    PrefillParams pp;
    const int32_t *prefix_lens;  // [num_seqs] or null
    int ctas;                    // CTAs of the cluster that takes a pair of tiles
    float near_max;              // raw scores up to this in size are capped by the polynomial
};

// =====================================================================================
// The query at position pos sees t if (t <= pos or t < prefix) and |pos - t| < window: one interval
// [lo, hi] that holds pos and moves up with it, so a 128-row tile needs the chunks of 128 keys from its first row's
// lo to its last row's hi, and a chunk that lies within all rows' intervals needs no mask.
//
// Roles and pipelines are those of prefill_tc_kernel (a CTA per pair of 128-row tiles, K and V chunks in two-stage
// rings, S and P in the same tensor-memory columns). What differs:
//  - each tile has its own first and last chunk; the pair walks their union, in which there is no gap;
//  - two warps clean values: a row that does not see a key must not meet its NaN or infinity (0 times either is NaN),
//    so in blocks that not every row sees such elements are zeroed before P V, and added at the end, element by
//    element, to the rows that see them;
//  - capped scores come from a polynomial, raw Q(raw^2) with Q that of cap tanh(y) / raw, y = raw scale / cap, for
//    |y| <= 3/4, 5.7e-7 of the score off. tanh by exponentials takes two more instructions a score on the
//    special-function unit, where a chunk's exponentials alone take as long as its products; only where a warp
//    holds a larger score among 64 columns are they taken that way.
//  - Weights come with their rounding remainders (a second P V) where a row may see few keys or give few all of
//    its weight: tiles with rows that see less than 64 keys, and with a bias by distance the chunks next to the tile's
//    positions and the first.
//
// Measured (32 q / 8 kv heads of 128, 512-token chunks behind 16K-32K tokens, 1.5 PFLOP; two CTAs to a pair): 1438 us with nothing
// transformed (1042 TFLOP/s; prefill_tc_kernel takes 1362), 1695 with a bias, 1868 capped at 50 (801 TFLOP/s), 2968 with
// scores past the polynomial. Per pair of tiles and chunk the MMAs take about 2500 clocks and the two
// softmaxes behind them 1900, 3250 with the cap, whose polynomial's six multiply-adds a score are most of the rest. Tried
// and slower, capped, where a CTA to a pair took 2035: the row unrolled in registers 2206; the same as one pass against the
// reference so far, redone where a score exceeds it by more than 2^8, 3020-3380; two threads to a row (sixteen warps)
// 2209; two 64-column S buffers a tile, so that products and softmax overlap, 2290 (2091 uncapped: products of 64
// columns take as long as of 128); the tiles' softmaxes in turns 2130, their first passes in turns 2038.
// Where pairs of tiles are few, a cluster of CTAs takes each: a CTA takes a run of the pair's chunks as if there were no
// others and leaves its rows' O, not yet divided, with their references and sums in its shared memory, whose rings are
// free by then; the cluster's CTAs then share the rows and join what all of them left through distributed shared memory.
// (16 tokens behind 16K, capped, 32 q / 8 kv heads of 128: 333 us with a CTA to a pair, 53 with eight.)
// 32 prompts of 64-2048 tokens, window 1024, capped: 720 us (594 uncapped); with one warp that cleans whole chunks 830, two
// 742, two that take only blocks with rows that are not seen 720.
// =====================================================================================
constexpr float kCapNear = 0.75f;
// tanh(y) / y = sum c_k y^2k, fitted on [0, kCapNear] (relative error 5.7e-7)
constexpr float kTanh0 = 0.999999435f, kTanh1 = -0.333282515f, kTanh2 = 0.132589832f, kTanh3 = -0.0500563012f,
                kTanh4 = 0.0129296311f;

// Up to which raw score the polynomial in powers of it holds. Every score is taken the long way where the cap is so
// small that its coefficients pass fp32. Where it is so large that they fall below fp32's normal numbers, scores from y = 1/20
// on are (to where c2 y^4 and what follows are below 2^-20), from 2^-12 on where c1 falls below too; and
// those whose square would pass fp32.
inline float capped_near_max(float scale_log2, float cap_in) {
    const double ci2 = (double)cap_in * cap_in, s = std::fabs((double)scale_log2);
    const double k1 = s * -kTanh1 * ci2, k4 = s * kTanh4 * ci2 * ci2 * ci2 * ci2;
    if (!(k4 <= FLT_MAX)) return -1.f;
    const double y = ci2 < FLT_MIN || k1 < FLT_MIN ? 0x1p-12 : k4 < FLT_MIN ? 0.05 : kCapNear;
    return cap_in == 0.f ? 0x1p60f : (float)std::min(y / std::fabs((double)cap_in), 0x1p60);
}

struct ScoredBars {
    uint64_t q_full;
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], v_clean[2];
    uint64_t s_full[2], p_full[2], o_done[2];  // per query tile
    uint64_t drain;
    uint32_t tmem_base;
    int any_bad;  // a value was not finite, and was zeroed
};
static_assert(sizeof(ScoredBars) <= 256, "barrier area");

// What a CTA of a cluster leaves of its pair of tiles, over the staging areas: O by row, padded so that threads with a row
// each write to different banks; and the rows' references and sums.
template <int D>
struct ScoredPart {
    static constexpr int kPitch = D + 4;
    float o[2][128][kPitch];
    float2 ml[2][128];
    static_assert(sizeof(float) * 2 * 128 * (kPitch + 2) <= TcCfg<D>::kBarOff, "staging areas");
};

// What a sequence's rows see.
struct Sight {
    int window, prefix;
    __device__ __forceinline__ int lo(int pos) const { return max(0, pos - window + 1); }
    __device__ __forceinline__ int hi(int pos) const {
        return min(max(pos, prefix - 1), pos - 1 + min(window, INT_MAX - pos));
    }
};

// One query tile: tokens t0 .. t_end - 1, chunks c0 .. c1 - 1, positions first .. last.
struct ScoredTile {
    int t0, t_end, c0, c1, first, last;
    // whether all rows see all of chunk j (128 keys), which lies before the sequence's last block
    __device__ __forceinline__ bool whole(const Sight &see, int j, int nblk) const {
        return (j + 1) * 8 < nblk && j * 128 >= see.lo(last) && j * 128 + 127 <= see.hi(first);
    }
    // whether its weights come with their remainders
    __device__ __forceinline__ bool split(const Sight &see, bool bias, int j) const {
        // (what a row sees grows with its position up to the window, and falls where the prefix' end stays ahead of it)
        const bool few = min(see.hi(first) - see.lo(first), see.hi(last) - see.lo(last)) < 63;
        return few || (bias && (j == c0 || (j >= first / 128 - 1 && j <= last / 128 + 1)));
    }
};

// Adds the values at positions [from, to] of a sequence that are not finite, columns d0 .. d0 + cols - 1, to those of a row
// that this thread has written (dst). Not in line: it is seldom called.
__device__ __noinline__ void scored_add_zeroed(const DecodeParams &p, int s, int h, int from, int to, int head_dim, int d0,
                                               int cols, __nv_bfloat16 *dst) {
#pragma unroll 1
    for (int ps = from; ps <= to; ++ps) {
        const int pb = __ldg(p.block_tables + (size_t)s * p.max_blocks_per_seq + ps / kBlock);
        if (pb < 0 || pb >= p.num_blocks) continue;
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v_cache) +
                                 (((size_t)pb * p.num_kv_heads + h) * kBlock + ps % kBlock) * head_dim + d0;
#pragma unroll 1
        for (int c = 0; c < cols; ++c) {
            const float x = __bfloat162float(v[c]);
            if (!(fabsf(x) < INFINITY)) dst[c] = __float2bfloat16_rn(__bfloat162float(dst[c]) + x);
        }
    }
}

// All threads of the cluster's CTAs, each of which comes here at the end of its bounded waits.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// Joins what the cluster's CTAs left of a pair of tiles that starts at token t0. Every CTA takes each ctas-th row, eight lanes
// to a row, so that a warp has the loads of four rows under way.
template <int D>
__device__ __noinline__ void scored_join(const DecodeParams &p, Sight see, ScoredPart<D> &part, int *any_bad, int ctas,
                                         int rank, int warp, int lane, int s, int h, int q0, int n, int t0, int tt,
                                         int first_pos) {
    namespace cg = cooperative_groups;
    constexpr int kVecs = D / 32;  // float4s of a lane: columns 4 sub + 32 v
    cg::cluster_group cluster = cg::this_cluster();
    const int g = p.group, tile_rows = tt * g, sub = lane & 7;
    const int rows = (min(n, t0 + 2 * tt) - t0) * g;  // of both tiles
    const int bad = sub < ctas ? *cluster.map_shared_rank(any_bad, sub) : 0;
#pragma unroll 1
    for (int base = rank + warp * 4 * ctas; base < rows; base += 32 * ctas) {
        const int i = base + (lane >> 3) * ctas;
        const bool mine = i < rows;
        const int t = mine && i >= tile_rows, row = mine ? i - t * tile_rows : 0;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (mine && sub < ctas) ml = cluster.map_shared_rank(&part, sub)->ml[t][row];
        float ms = ml.x;
#pragma unroll
        for (int d = 4; d; d >>= 1) ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, d));
        const float w = ex2_approx(ml.x - (ms == -INFINITY ? 0.f : ms));
        float l = 0.f;
        float4 o[kVecs] = {};
#pragma unroll 2
        for (int r = 0; r < ctas; ++r) {
            const float wr = __shfl_sync(0xffffffffu, w, r, 8), lr = __shfl_sync(0xffffffffu, ml.y, r, 8);
            if (lr == 0.f) continue;  // the row saw nothing there
            l = fmaf(wr, lr, l);
            const float4 *src = reinterpret_cast<const float4 *>(cluster.map_shared_rank(&part, r)->o[t][row]) + sub;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const float4 x = src[v * 8];
                o[v] = make_float4(fmaf(wr, x.x, o[v].x), fmaf(wr, x.y, o[v].y), fmaf(wr, x.z, o[v].z), fmaf(wr, x.w, o[v].w));
            }
        }
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // (NaN stays)
        const int token = t0 + i / g, head = h * g + i % g;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + ((size_t)(q0 + token) * p.num_q_heads + head) * D + sub * 4;
        if (mine)
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const __nv_bfloat162 a = __floats2bfloat162_rn(o[v].x * inv, o[v].y * inv);
                const __nv_bfloat162 c = __floats2bfloat162_rn(o[v].z * inv, o[v].w * inv);
                *reinterpret_cast<uint2 *>(dst + v * 32) =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&c));
            }
        // what was zeroed shows in its element of the rows that see it (what was not shows already)
        if (__builtin_expect(__any_sync(0xffffffffu, bad != 0), 0) && mine)
            for (int v = 0; v < kVecs; ++v)
                scored_add_zeroed(p, s, h, see.lo(first_pos + token), see.hi(first_pos + token), D, sub * 4 + v * 32, 4,
                                  dst + v * 32);
    }
}

// kCap, kBias: whether scores are capped and biased.
template <int D, bool kCap, bool kBias>
__global__ void __launch_bounds__(TcCfg<D>::kThreads, 1)
    prefill_scored_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const ScoredPrefillParams sp) {
    using C = TcCfg<D>;
    const PrefillParams &pp = sp.pp;
    const DecodeParams &p = pp.d;
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctas = sp.ctas, h = blockIdx.x / ctas, rank = blockIdx.x - h * ctas;
    int s, pair;
    if (pp.seq_major) {
        pair = gridDim.y - 1 - blockIdx.y;
        s = prefill_sequence_by_rank(pp, blockIdx.z, tid);
    } else {
        s = blockIdx.y;
        pair = gridDim.z - 1 - blockIdx.z;
    }
    const bool flagger = blockIdx.x == 0 && pair == 0;  // one CTA per sequence reports bad lengths
    const int g = p.group;
    const int q0 = __ldg(pp.query_start + s);
    const long long nn = (long long)__ldg(pp.query_start + s + 1) - q0;
    const int len = seq_len(p, s, tid == 0 && flagger);
    const int tt = pp.tile_tokens;
    Sight see{p.window, sp.prefix_lens ? __ldg(sp.prefix_lens + s) : 0};
    if (see.prefix < 0 && tid == 0 && flagger) raise_error(PKV_DEVERR_LENGTH);
    see.prefix = min(max(see.prefix, 0), len);
    if (nn < 0 || nn > len || nn > pp.max_query_len || q0 < 0 || q0 + nn > pp.num_queries) {
        if (tid == 0 && flagger) raise_error(PKV_DEVERR_LENGTH);
        return;  // (the whole cluster, as below)
    }
    const int n = (int)nn;
    if (pair * C::kTiles * tt >= n) return;
    const int first_pos = len - n;  // position of new token 0
    ScoredTile tl[C::kTiles];
#pragma unroll
    for (int t = 0; t < C::kTiles; ++t) {
        ScoredTile &x = tl[t];
        x.t0 = (pair * C::kTiles + t) * tt;
        x.t_end = min(n, x.t0 + tt);
        x.first = first_pos + x.t0;
        x.last = first_pos + x.t_end - 1;
        if (x.t0 < n) {
            x.c0 = see.lo(x.first) / C::kKeys;
            x.c1 = see.hi(x.last) / C::kKeys + 1;
        } else {
            x.c0 = x.c1 = tl[0].c1;  // (an empty second tile)
        }
    }
    int j0 = tl[0].c0, j1 = max(tl[0].c1, tl[1].c1);
    if (ctas > 1) {  // this CTA's run of the chunks, which may be empty
        const int chunks = j1 - j0, from = j0;
        j0 = from + (int)((long long)chunks * rank / ctas);
        j1 = from + (int)((long long)chunks * (rank + 1) / ctas);
#pragma unroll
        for (int t = 0; t < C::kTiles; ++t) {
            tl[t].c0 = min(max(tl[t].c0, j0), j1);
            tl[t].c1 = max(min(tl[t].c1, j1), tl[t].c0);
        }
    }
    const int nblk = (len + kBlock - 1) / kBlock;
    const int last_valid = len - (nblk - 1) * kBlock;
    const int first_blk = see.lo(tl[0].first) / kBlock;  // blocks before it are not read

    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    ScoredBars &b = *reinterpret_cast<ScoredBars *>(base + C::kBarOff);
    if (tid == 0) {
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        mbar_init(&b.q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.k_full[i], 1);
            mbar_init(&b.k_empty[i], 1);
            mbar_init(&b.v_full[i], 1);
            mbar_init(&b.v_empty[i], 1);
            mbar_init(&b.v_clean[i], 2);
            mbar_init(&b.s_full[i], 1);
            mbar_init(&b.p_full[i], 4);
            mbar_init(&b.o_done[i], 1);
        }
        mbar_init(&b.drain, 1);
        b.any_bad = 0;
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(&b.tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem_base;
    const uint32_t q_s = smem_u32(base + C::kQOff), k_s = smem_u32(base + C::kKOff);
    const uint32_t v_s = smem_u32(base + C::kVOff);
    auto active = [&](int t, int j) { return j >= tl[t].c0 && j < tl[t].c1; };
    if (warp < 4) {
      setmaxnreg_dec<C::kLowRegs>();
      if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0 && j0 < j1) {
            bool ok = true;
            int qbytes = 0;
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) qbytes += tl[t].t0 < n ? C::kHalves * 128 * g * tt : 0;
            mbar_arrive_expect_tx(&b.q_full, qbytes);
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t)
                if (tl[t].t0 < n)
                    for (int u = 0; u < C::kHalves; ++u)
                        tma_load_4d(base + C::kQOff + t * C::kQBytes + u * C::kHalfRows, &tmq, 0, u, h * g,
                                    q0 + tl[t].t0, &b.q_full);
            const int32_t *table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
            int issued_k = 0, issued_v = 0;  // chunks whose K / V copies were issued
            for (int j = j0; j < j1 && ok; ++j) {
                const int r = j - j0, st = r & 1;
                if (r >= 2 && !mbar_wait(&b.k_empty[st], ((r - 2) >> 1) & 1)) {
                    ok = false;
                    break;
                }
                // the chunk's blocks: tile row z of the cache view (-1, outside the tensor, reads as zeros: not
                // seen by any row, past the sequence, or a bad id) and first slot y
                int z[C::kChunkBlocks], y[C::kChunkBlocks];
#pragma unroll
                for (int bi = 0; bi < C::kChunkBlocks; ++bi) {
                    const int blk = j * C::kChunkBlocks + bi;
                    z[bi] = blk >= first_blk && blk < nblk ? __ldg(table + blk) : -1;
                }
#pragma unroll
                for (int bi = 0; bi < C::kChunkBlocks; ++bi) {
                    const int blk = j * C::kChunkBlocks + bi;
                    y[bi] = blk == nblk - 1 ? last_valid - kBlock : 0;
                    if (blk >= first_blk && blk < nblk) {
                        if (z[bi] < 0 || z[bi] >= p.num_blocks) {
                            raise_error(PKV_DEVERR_BLOCK_ID);
                            z[bi] = -1;
                        } else {
                            z[bi] = z[bi] * p.num_kv_heads + h;
                        }
                    }
                }
                // K chunk as [half][128 keys][64]: 8-row groups 1024 bytes apart along the keys
                mbar_arrive_expect_tx(&b.k_full[st], C::kStage);
#pragma unroll
                for (int bi = 0; bi < C::kChunkBlocks; ++bi)
#pragma unroll
                    for (int u = 0; u < C::kHalves; ++u)
                        tma_load_4d(base + C::kKOff + st * C::kStage + u * C::kHalfRows + bi * (kBlock * 128), &tmk,
                                    0, y[bi], u, z[bi], &b.k_full[st]);
                issued_k = r + 1;
                if (r >= 2 && !mbar_wait(&b.v_empty[st], ((r - 2) >> 1) & 1)) {
                    ok = false;
                    break;
                }
                // V chunk as [block][half][16 keys][64]
                mbar_arrive_expect_tx(&b.v_full[st], C::kStage);
#pragma unroll
                for (int bi = 0; bi < C::kChunkBlocks; ++bi)
                    tma_load_4d(base + C::kVOff + st * C::kStage + bi * C::kBlockBytes, &tmv, 0, y[bi], 0, z[bi],
                                &b.v_full[st]);
                issued_v = r + 1;
            }
            if (!ok) raise_error(PKV_DEVERR_TIMEOUT);
            // no copy may land after the CTA is gone: wait (bounded) for the last one of each stage
            for (int r = max(0, issued_k - 2); r < issued_k; ++r) mbar_wait(&b.k_full[r & 1], (r >> 1) & 1);
            for (int r = max(0, issued_v - 2); r < issued_v; ++r) mbar_wait(&b.v_full[r & 1], (r >> 1) & 1);
            mbar_wait(&b.q_full, 0);
        }
      } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        if (lane == 0 && j0 < j1) {
            constexpr uint32_t idesc_s = idesc_bf16_f32(C::kRows, C::kKeys, false, false);
            constexpr uint32_t idesc_o = idesc_bf16_f32(C::kRows, D, false, true);
            auto issue_s = [&](int t, int r) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {  // 16 head-dim elements per step
                    const uint32_t off = (kk >> 2) * C::kHalfRows + (kk & 3) * 32;
                    umma_bf16(tmem + t * C::kTileCols, smem_desc_sw128(q_s + t * C::kQBytes + off, 16, 1024),
                              smem_desc_sw128(k_s + (r & 1) * C::kStage + off, 16, 1024), idesc_s, kk > 0);
                }
            };
            auto issue_pv = [&](int t, int r, bool start, bool split) {
#pragma unroll
                for (int kk = 0; kk < C::kChunkBlocks; ++kk) {  // 16 keys (one block) per step
                    const uint64_t vd =
                        smem_desc_sw128(v_s + (r & 1) * C::kStage + kk * C::kBlockBytes, kBlock * 128, 1024);
                    // P of keys 16 kk .. 16 kk + 15: columns 32 (kk / 2) + 8 (kk % 2); remainder 16 further
                    const uint32_t pa = tmem + t * C::kTileCols + (kk >> 1) * 32 + (kk & 1) * 8;
                    umma_bf16_tmem_a(tmem + t * C::kTileCols + C::kOCol, pa, vd, idesc_o, !start || kk > 0);
                    if (split) umma_bf16_tmem_a(tmem + t * C::kTileCols + C::kOCol, pa + 16, vd, idesc_o, true);
                }
            };
            bool ok = mbar_wait(&b.q_full, 0) && mbar_wait(&b.k_full[0], 0);
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < C::kTiles; ++t)
                    if (active(t, j0)) {
                        issue_s(t, 0);
                        umma_commit(&b.s_full[t]);
                    }
                umma_commit(&b.k_empty[0]);
            }
            for (int j = j0; ok && j < j1; ++j) {
                const int r = j - j0;
                ok = mbar_wait(&b.v_clean[r & 1], (r >> 1) & 1);
                if (ok && j + 1 < j1) ok = mbar_wait(&b.k_full[(r + 1) & 1], ((r + 1) >> 1) & 1);
                if (!ok) break;
#pragma unroll
                for (int t = 0; t < C::kTiles; ++t) {
                    const bool now = active(t, j), next = active(t, j + 1);
                    if (now) {
                        if (!(ok = mbar_wait(&b.p_full[t], (j - tl[t].c0) & 1))) break;
                        tc_fence_after();
                        issue_pv(t, r, j == tl[t].c0, tl[t].split(see, kBias, j));
                        if (!next) umma_commit(&b.o_done[t]);
                    }
                    if (next) {
                        tc_fence_after();
                        issue_s(t, r + 1);
                        umma_commit(&b.s_full[t]);
                    }
                }
                if (!ok) break;
                umma_commit(&b.v_empty[r & 1]);
                if (j + 1 < j1) umma_commit(&b.k_empty[(r + 1) & 1]);
            }
            if (!ok) raise_error(PKV_DEVERR_TIMEOUT);
            // every MMA issued has finished before the tensor memory is released
            umma_commit(&b.drain);
            mbar_wait(&b.drain, 0);
        }
        __syncwarp();
      } else {
        // ------------------------------ values that not every row sees ------------------------------
        bool ok = true;
        for (int j = j0; j < j1 && ok; ++j) {
            const int r = j - j0, st = r & 1;
            if (!(ok = warp_wait(&b.v_full[st], (r >> 1) & 1))) break;
            // blocks with positions that some row does not see: before `low` and after `high`
            int low = INT_MIN, high = INT_MAX;
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t)
                if (active(t, j)) {
                    if (tl[t].split(see, kBias, j)) low = INT_MAX;  // (a remainder may be negative: the whole chunk)
                    low = max(low, see.lo(tl[t].last));
                    high = min(high, see.hi(tl[t].first));
                }
            const int blk0 = j * C::kChunkBlocks, blocks = min(C::kChunkBlocks, nblk - blk0);
            const int upto = low > blk0 * kBlock ? min(blocks, (min(low, len) - 1) / kBlock + 1 - blk0) : 0;
            const int from = high < len ? max(upto, (high + 1) / kBlock - blk0) : blocks;
            uint8_t *vst = base + C::kVOff + st * C::kStage;
            constexpr int kVecs = C::kBlockBytes / 16;
            auto clean = [&](int b_lo, int b_hi) {
#pragma unroll 1
                for (int i = b_lo * kVecs + (warp - 2) * 32 + lane; i < b_hi * kVecs; i += 64) {
                    const uint4 v = reinterpret_cast<const uint4 *>(vst)[i];
                    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                    uint32_t bad[4];  // the top bit of each half whose exponent is all ones
#pragma unroll
                    for (int e = 0; e < 4; ++e) bad[e] = ((x[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                    if ((bad[0] | bad[1]) | (bad[2] | bad[3])) {
                        uint32_t keep[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            keep[e] = (bad[e] & 0x8000u ? 0u : 0xffffu) | (bad[e] & 0x80000000u ? 0u : 0xffff0000u);
                        reinterpret_cast<uint4 *>(vst)[i] =
                            make_uint4(x[0] & keep[0], x[1] & keep[1], x[2] & keep[2], x[3] & keep[3]);
                        *reinterpret_cast<volatile int *>(&b.any_bad) = 1;
                    }
                }
            };
            if (upto > 0 || from < blocks) {
                clean(0, upto);
                clean(from, blocks);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.v_clean[st]);
        }
        if (!ok && lane == 0) raise_error(PKV_DEVERR_TIMEOUT);
      }
      if (ctas > 1) {
          __syncwarp();
          cluster_barrier();
      }
    } else {
        setmaxnreg_inc<C::kHighRegs>();
        // ------------------------------ softmax ------------------------------
        const int t = (warp - 4) >> 2;  // query tile
        const int quad = warp & 3;       // tensor-memory lanes 32 quad .. 32 quad + 31
        const int row = quad * 32 + lane;
        static_assert(C::kTiles == 2, "tile selection below");
        const ScoredTile me = {t ? tl[1].t0 : tl[0].t0, t ? tl[1].t_end : tl[0].t_end, t ? tl[1].c0 : tl[0].c0,
                               t ? tl[1].c1 : tl[0].c1, t ? tl[1].first : tl[0].first, t ? tl[1].last : tl[0].last};
        const int rows = me.t0 < n ? (me.t_end - me.t0) * g : 0;
        const bool row_ok = row < rows;
        const int row_token = row / g, row_head = row - row_token * g;
        const int pos = me.first + (row_ok ? row_token : 0);
        const int lo_t = see.lo(pos), hi_t = see.hi(pos);  // (rows past the tile's end see what its first does)
        const uint32_t cols = tmem + ((uint32_t)(quad * 32) << 16) + t * C::kTileCols;
        const float slope = kBias ? slope_log2(p.slopes, h * g + row_head, p.num_q_heads) : 0.f;
        // the polynomial's coefficients in powers of the raw score (capped_near_max)
        const float ci2 = p.cap_in * p.cap_in;
        const float k0 = kCap ? p.scale_log2 * kTanh0 : p.scale_log2, k1 = p.scale_log2 * kTanh1 * ci2;
        const float k2 = p.scale_log2 * kTanh2 * ci2 * ci2, k3 = p.scale_log2 * kTanh3 * ci2 * ci2 * ci2;
        const float k4 = p.scale_log2 * kTanh4 * ci2 * ci2 * ci2 * ci2;
        // Without either scores stay raw: x sl is the log2-domain score, the sign is folded in; a scale of 0 becomes one
        // that leaves every score 0, so that a masked -inf stays -inf.
        const float sl = kCap || kBias ? 1.f : fmaxf(fabsf(p.scale_log2), 1e-30f);
        const uint64_t f0 = pack_f2(k0, k0), f1 = pack_f2(k1, k1), f2 = pack_f2(k2, k2), f3 = pack_f2(k3, k3);
        const uint64_t f4 = pack_f2(k4, k4), zero = pack_f2(0.f, 0.f), sl2 = pack_f2(sl, sl);
        const uint64_t slope2 = pack_f2(slope, slope), two = pack_f2(2.f, 2.f);
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = me.c0; j < me.c1; ++j) {
            if (!(ok = warp_wait(&b.s_full[t], (j - me.c0) & 1))) break;
            tc_fence_after();
            const bool whole = me.whole(see, j, nblk), split = me.split(see, kBias, j);
            // Columns kc = 0 .. 127: a full block's column holds position c0 + kc; in the chunk with the sequence's last
            // block, which was loaded `early` rows early, column kc >= cut holds position c0 + kc - early and is a token
            // from cut + early on. So a row sees columns a0 .. a1 and b0 .. b1.
            const int c0 = j * C::kKeys, cut = (nblk - 1) * kBlock - c0, early = kBlock - last_valid;
            // the bias is linear in the column unless there are keys behind the query, or shifted ones
            const bool bent = kBias && ((see.prefix - 1 > me.first && c0 + 127 > me.first) || (cut < 128 && early > 0));
            const uint64_t at2 = pack_f2((float)(c0 - pos) * slope, (float)(c0 - pos) * slope);
            // scores of a pair of columns from raw ones, in registers; col: the pair's columns
            auto near = [&](uint64_t r, uint64_t col) -> uint64_t {
                uint64_t f = f0;
                if constexpr (kCap) {
                    const uint64_t r2 = fma_f2(r, r, zero);
                    f = fma_f2(fma_f2(fma_f2(fma_f2(f4, r2, f3), r2, f2), r2, f1), r2, f0);
                }
                return fma_f2(r, f, kBias ? fma_f2(col, slope2, at2) : zero);
            };
            // Two rolled passes over the row, 64 columns at a time: scores and their maximum, then weights. One or two warps a
            // scheduler run this code, and its fetching counts.
            const int a0 = lo_t - c0, a1 = min(hi_t - c0, cut - 1);
            const int b0 = max(cut, a0) + early, b1 = hi_t - c0 + early;
            const float mid = (float)(pos - c0);
            const bool rewrite = kCap || kBias || !whole || p.scale_log2 < 0.f;
            float mx = -INFINITY;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                float v[2][32];
                const uint32_t hc = cols + half * 64;
                tmem_ld32(hc, v[0]);
                tmem_ld32(hc + 32, v[1]);
                tmem_wait_ld();
                bool far = bent;
                if constexpr (kCap) {
                    float big[2] = {0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int e = 0; e < 32; e += 2) big[q] = max3f(big[q], fabsf(v[q][e]), fabsf(v[q][e + 1]));
                    far |= __any_sync(0xffffffffu, row_ok && !(fmaxf(big[0], big[1]) <= sp.near_max));
                }
                if ((kCap || kBias) && __builtin_expect(far, 0)) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int kc = half * 64 + q * 32 + e;
                            v[q][e] = kCap ? capped(v[q][e], p.cap_in, p.cap_log2) : v[q][e] * p.scale_log2;
                            if constexpr (kBias) v[q][e] = fmaf(-slope, fabsf(mid - (kc >= cut ? kc - early : kc)), v[q][e]);
                        }
                } else if constexpr (kCap || kBias) {
                    uint64_t col = pack_f2((float)(half * 64), (float)(half * 64 + 1));
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            unpack_f2(near(pack_f2(v[q][e], v[q][e + 1]), col), v[q][e], v[q][e + 1]);
                            if constexpr (kBias) col = add_f2(col, two);
                        }
                } else if (__builtin_expect(p.scale_log2 < 0.f, 0)) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[q][e] = -v[q][e];
                }
                if (!whole) {
                    auto upto = [](int c) { return c < 0 ? 0u : c >= 31 ? ~0u : (2u << c) - 1; };  // columns 0 .. c
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int o = half * 64 + q * 32;
                        const uint32_t bits = (upto(a1 - o) & ~upto(a0 - 1 - o)) | (upto(b1 - o) & ~upto(b0 - 1 - o));
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[q][e] = bits & (1u << e) ? v[q][e] : -INFINITY;
                    }
                }
                float mxs[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int e = 0; e < 32; e += 2) mxs[(e >> 1) & 3] = max3f(mxs[(e >> 1) & 3], v[q][e], v[q][e + 1]);
                mx = fmaxf(max3f(mxs[0], mxs[1], mxs[2]), mxs[3]);
                if (rewrite) {
                    tmem_st32(hc, v[0]);
                    tmem_st32(hc + 32, v[1]);
                }
            }
            const float m_new = fmaxf(m, mx * sl);
            const bool move = m_new > m + 8.f;
            const float m_use = move ? m_new : m;
            const float ms = m_use == -INFINITY ? 0.f : m_use;
            const float alpha = ex2_approx(m - ms);
            if (rewrite) tmem_wait_st();
            // this tile's O is quiescent here (P V of the previous chunk ran before S of this one)
            if (__builtin_expect(j > me.c0 && __any_sync(0xffffffffu, row_ok && move && m != -INFINITY), 0)) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(cols + C::kOCol + c * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] *= alpha;
                    tmem_st32(cols + C::kOCol + c * 32, o);
                }
            }
            m = m_use;
            l *= alpha;
            const uint64_t nms2 = pack_f2(-ms, -ms);
            uint64_t rss[4] = {zero, zero, zero, zero};
            auto weights = [&](auto split_c) {
                constexpr bool kSplit = decltype(split_c)::value;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    float v[2][32];
                    const uint32_t hc = cols + half * 64;
                    tmem_ld32(hc, v[0]);
                    tmem_ld32(hc + 32, v[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t hi[16], rem[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float e0, e1;
                            const uint64_t y = pack_f2(v[q][2 * i], v[q][2 * i + 1]);
                            unpack_f2(kCap || kBias ? add_f2(y, nms2) : fma_f2(y, sl2, nms2), e0, e1);
                            e0 = ex2_approx(e0);
                            e1 = ex2_approx(e1);
                            rss[i & 3] = add_f2(rss[i & 3], pack_f2(e0, e1));
                            const __nv_bfloat162 ph = __floats2bfloat162_rn(e0, e1);
                            hi[i] = *reinterpret_cast<const uint32_t *>(&ph);
                            if constexpr (kSplit) {
                                const __nv_bfloat162 pl = __floats2bfloat162_rn(
                                    e0 - __uint_as_float(hi[i] << 16), e1 - __uint_as_float(hi[i] & 0xffff0000u));
                                rem[i] = *reinterpret_cast<const uint32_t *>(&pl);
                            }
                        }
                        tmem_st16(hc + q * 32, hi);
                        if constexpr (kSplit) tmem_st16(hc + q * 32 + 16, rem);
                    }
                }
            };
            if (__builtin_expect(split, 0)) weights(BoolConst<true>{});
            else weights(BoolConst<false>{});
            float r[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack_f2(rss[i], r[2 * i], r[2 * i + 1]);
            l += ((r[0] + r[1]) + (r[2] + r[3])) + ((r[4] + r[5]) + (r[6] + r[7]));
            // P = 2^(x sl - reference) in bf16 lies over each quarter's own score columns: keys 32 q + 2 i, + 1 at column
            // 32 q + i, their rounding remainders at + 16. The row sum takes the unrounded weights.
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.p_full[t]);
        }
        if (ctas > 1) {
            // both tiles are through with the staging areas
#pragma unroll
            for (int u = 0; u < C::kTiles; ++u)
                if (ok && tl[u].c0 < tl[u].c1) ok = warp_wait(&b.o_done[u], 0);
            if (!ok) raise_error(PKV_DEVERR_TIMEOUT);
            tc_fence_after();
            ScoredPart<D> &part = *reinterpret_cast<ScoredPart<D> *>(base);
            const bool some = ok && me.c0 < me.c1;
            if (row_ok) part.ml[t][row] = some ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
            if (some) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(cols + C::kOCol + c * 32, o);
                    tmem_wait_ld();
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(&part.o[t][row][c * 32 + e]) =
                                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
            }
            cluster_barrier();
            scored_join<D>(p, see, part, &b.any_bad, ctas, rank, warp - 4, lane, s, h, q0, n, tl[0].t0, tt, first_pos);
        } else if (me.t0 < n) {
            if (ok) ok = warp_wait(&b.o_done[t], 0);
            if (!ok) {
                raise_error(PKV_DEVERR_TIMEOUT);
            } else {
                tc_fence_after();
                const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // (NaN stays)
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                     ((size_t)(q0 + me.t0 + (row_ok ? row_token : 0)) * p.num_q_heads + h * g + row_head) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(cols + C::kOCol + c * 32, o);
                    tmem_wait_ld();
                    if (row_ok) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 v2 = __floats2bfloat162_rn(o[q * 8 + 2 * e] * inv,
                                                                                o[q * 8 + 2 * e + 1] * inv);
                                w[e] = *reinterpret_cast<const uint32_t *>(&v2);
                            }
                            *reinterpret_cast<uint4 *>(dst + c * 32 + q * 8) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (__builtin_expect(*reinterpret_cast<volatile int *>(&b.any_bad) != 0, 0) && row_ok) {
                    // what was zeroed shows in its element of the rows that see it, whatever its weight
                    for (int j = me.c0; j < me.c1; ++j) {
                        bool clean = false;
#pragma unroll
                        for (int u = 0; u < C::kTiles; ++u)
                            clean |= active(u, j) && (!tl[u].whole(see, j, nblk) || tl[u].split(see, kBias, j));
                        if (clean)
                            scored_add_zeroed(p, s, h, max(lo_t, j * C::kKeys), min(hi_t, j * C::kKeys + C::kKeys - 1), D,
                                              0, D, dst);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (ctas > 1) cluster_barrier();  // no CTA leaves while others read what it left
}

}  // namespace pkv
