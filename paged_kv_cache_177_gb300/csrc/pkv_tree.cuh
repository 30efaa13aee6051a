// pkv_tree.cuh -- drafted tokens: the mask of a tree from its parents,
// attention of a tree's rows over the paged cache, and the move of the
// accepted path's keys and values to consecutive positions.
#pragma once

#include "pkv_prefill_tc.cuh"

namespace pkv {

struct TreeParams {
    DecodeParams d;              // context_lens count the drafts
    const int32_t *query_start;  // [num_seqs + 1]
    const int64_t *mask;         // [num_queries][mask_words]
    int mask_words, num_queries, max_query_len;
};

// A sequence's first row and number of drafts; false (flagged by the caller's
// choice of thread) if they do not fit the context or the arrays.
__device__ __forceinline__ bool tree_rows(const int32_t *query_start, int s, int len, int max_query_len,
                                          int num_queries, int &q0, int &n) {
    q0 = __ldg(query_start + s);
    const long long nn = (long long)__ldg(query_start + s + 1) - q0;
    n = (int)nn;
    return nn >= 0 && nn <= len && nn <= max_query_len && q0 >= 0 && q0 + nn <= num_queries;
}

// =====================================================================================
// Masks from parents: one thread per draft walks up. Parents come before their children, so
// the walk meets falling indexes and fills the row's words from the last to the first. Its time is the deepest draft's
// chain of loads, and a thread's drafts are 64 apart: 64 sequences of 32 drafts 2.5 us (4.6 as chains), 8 of 256 17 us
// (68 as chains), one of 1024 217 us and, as one chain, 990 us.
// =====================================================================================
__global__ void tree_masks_kernel(int64_t *mask, const int32_t *parents, const int32_t *query_start, int num_queries,
                                  int max_query_len, int words) {
    const int s = blockIdx.x;
    int q0, n;
    if (!tree_rows(query_start, s, INT_MAX, max_query_len, num_queries, q0, n)) {
        if (threadIdx.x == 0) raise_error(PKV_DEVERR_LENGTH);
        return;
    }
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        unsigned long long *row = reinterpret_cast<unsigned long long *>(mask) + (size_t)(q0 + i) * words;
        int w = words - 1;
        unsigned long long bits = 0;
        for (int j = i; j >= 0;) {
            for (; w > j / 64; --w) {
                row[w] = bits;
                bits = 0;
            }
            bits |= 1ull << (j % 64);
            const int up = __ldg(parents + q0 + j);
            if (up < -1 || up >= j) {
                raise_error(PKV_DEVERR_INDEX);
                break;
            }
            j = up;
        }
        for (; w >= 0; --w) {
            row[w] = bits;
            bits = 0;
        }
    }
}

// =====================================================================================
// Attention on the 5th-generation tensor cores (tcgen05).
//
// Rows are (draft, query head of the kv head's group) pairs, 128 to an MMA tile (128 / g drafts), keys
// are taken 128 at a time (8 cache blocks, a chunk). All (sequence, kv head, row set) units' chunks form
// one line of T positions, cut into equal ranges, one per CTA (one CTA per SM), so every SM
// streams the same bytes whatever the lengths; a unit cut by a range's end leaves one state per
// segment -- row max (log2 domain), sum and unnormalised output, fp32 -- that tree_merge_kernel
// joins. Contexts of a few chunks are not cut: a CTA then takes whole units.
//
// The work of a drafts' batch is to read the context once: 4 D bytes of K and V a token and
// kv head, against 4 D flops per row, so up to about 256 rows HBM bounds it, and the roles below are
// there to keep 64 to 190 KB of copies in flight per SM:
//   warps 0 and 2        TMA: a unit's Q rows and the K chunks; the V chunks (two warps, so that neither
//                        ring waits for the other's stages)
//   warp 1, one thread   MMA: S = Q K^T (128 x 128, fp32 in tensor memory); O += P V with P from tensor memory
//   warp 3               the values of the drafts: a row that does not see a draft must not meet its
//                        NaN or infinity (0 times either is NaN), so such elements are zeroed before P V and
//                        added at the end, by element, to the rows that see them. (Of the context too where
//                        weights come with remainders, which are zero or negative as well.)
//   warps 4-7, 8-11      softmax, one thread per row (tensor-memory lane): two sides
// The two sides are two row tiles of a unit (kPair, units of more than 128 rows), or take turns at the
// chunks of one tile, each with its own S, O and running max; their two states are joined, half
// of the columns each, when the segment ends. Either way one side's softmax runs while the tensor
// cores work for the other.
//
// A row's max moves only when it grows by more than 8 (log2), as in the prefill kernels, and as there the
// weights of rows that may see few keys enter P V as two bf16 values, the rounded weight and its
// remainder (16 significant bits): such a row would carry the full rounding of its weights. These are the
// sequences of less than kPrefillSplitPositions context tokens, in all of their chunks: a draft far down a
// wide tree may see itself and a few others only. Over more keys the roundings average out, to about the
// output's own (the remainder everywhere takes 97 us on 64 sequences of up to 32 drafts, 32 q / 8 kv heads, where 75 do,
// and 397 us on eight contexts of 32K-128K, 16 drafts, 8 heads to a kv head, where 339 do).
//
// Every wait is bounded; on a timeout the role records PKV_DEVERR_TIMEOUT, waits (bounded) for its own
// copies and MMAs in flight, and the CTA frees its tensor memory and exits.
// =====================================================================================
template <int D, bool kPair>
struct TreeCfg {
    static constexpr int kRows = 128, kSides = 2;
    static constexpr int kTiles = kPair ? 2 : 1;           // row tiles of a unit
    static constexpr int kUnitRows = kTiles * kRows;
    static constexpr int kKeys = 128, kChunkBlocks = kKeys / kBlock;
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfRows = 128 * 128;            // bytes of 128 rows of 128 bytes
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kStage = kKeys * D * 2;           // one chunk of K (or of V)
    static constexpr int kBlockBytes = kBlock * D * 2;
    static constexpr int kStages = D == 128 ? (kPair ? 2 : 3) : 4;
    static constexpr int kKOff = kTiles * kQBytes;
    static constexpr int kVOff = kKOff + kStages * kStage;
    static constexpr int kBarOff = kVOff + kStages * kStage;
    static constexpr int kBarBytes = 512;
    static constexpr int kXchOff = kBarOff + kBarBytes;    // [2 sides][128 rows] (max, sum)
    static constexpr int kSmem = kXchOff + (kPair ? 0 : kSides * kRows * 8);
    static constexpr int kThreads = 384;
    static constexpr int kLowRegs = 104, kHighRegs = 200;   // setmaxnreg split, launched at 168
    static_assert(128 * kLowRegs + 256 * kHighRegs <= kThreads * 168, "register split");
    static constexpr uint32_t kTmemCols = 512, kSideCols = 256, kOCol = 128;
};

struct TreeBars {
    uint64_t q_full, q_empty;
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t v_clean[4];                       // per stage: its drafts' values are finite
    uint64_t s_full[2], p_full[2], o_done[2];  // per side
    uint64_t x_full[2], x_done[2];             // per side: its state is in shared memory; it has read both O
    uint64_t drain;
    uint32_t tmem_base;
    int any_bad;                                // a value was not finite, and was zeroed
    int start_seq;                              // where this CTA's range begins: sequence ...
    long long start_in;                         // ... position within the sequence, ...
    int start_rows[3];                          // ... its length, first row and drafts,
    long long total;                            // and the line's length
    long long warp_sum[12];
};
static_assert(sizeof(TreeBars) <= 512, "barrier area");

// A unit cut by the end of a worker's range: its segments (0: not cut), and where its rows go.
struct TreeCut {
    int segments, q_row, drafts, head;  // first query row of the unit, its drafts, first query head
};

// Whether a unit's weights come with their remainders: where a row may see fewer than 64 keys.
__device__ __forceinline__ bool tree_split(int ctx) { return ctx < kPrefillSplitPositions; }

// The first position whose values are cleaned before P V: the drafts', which not every row sees, and all that a
// remainder meets.
__device__ __forceinline__ int tree_first_clean(int ctx) { return tree_split(ctx) ? 0 : ctx; }

// The line that is cut into the workers' ranges: every unit takes kTreeUnitCost positions for its start and end (Q, a
// masked chunk, the join of the sides, the output: about as long as that many chunks), then one per chunk.
// (64 sequences, 32 q / 8 kv heads: 75 us, 90 with no cost, 83 with one, 82 with six; 13B-class: 303, 385, 321, 332.)
// A worker does the chunks whose positions lie in its range; where units are not to be cut, those whose
// start does.
constexpr int kTreeUnitCost = 3;

// How many workers a line of T positions gets.
__device__ __forceinline__ int tree_workers(long long T) { return (int)min((long long)gridDim.x, max(1LL, T / 4)); }

// A worker's way along the line: one segment (a unit's chunks c0 .. c1 - 1) at a time.
template <int D, bool kPair>
struct TreeWalk {
    using C = TreeCfg<D, kPair>;
    int s, unit, units;       // sequence, unit within it (kv head major, then row set), its units
    int len, q0, n, chunks, sets;
    int c0, c1;
    long long x, end;         // position of the unit's start; end of the worker's range

    // Positions of sequence s; flag: whether this call reports bad lengths and row counts.
    __device__ __forceinline__ static long long weigh(const TreeParams &tp, int s, int per_set, bool flag, int &len,
                                                int &q0, int &n) {
        len = seq_len(tp.d, s, flag);
        if (!tree_rows(tp.query_start, s, len, tp.max_query_len, tp.num_queries, q0, n)) {
            if (flag) raise_error(PKV_DEVERR_LENGTH);
            n = 0;
        }
        const int sets = (n + per_set - 1) / per_set;
        return (long long)sets * tp.d.num_kv_heads * ((len + C::kKeys - 1) / C::kKeys + kTreeUnitCost);
    }
    __device__ __forceinline__ void enter(const TreeParams &tp, int per_set) {  // the sequence s
        weigh(tp, s, per_set, false, len, q0, n);
        derive(tp, per_set);
    }
    __device__ __forceinline__ void derive(const TreeParams &tp, int per_set) {
        sets = (n + per_set - 1) / per_set;
        units = sets * tp.d.num_kv_heads;
        chunks = (len + C::kKeys - 1) / C::kKeys;
    }
    // To the unit after this one; false past the end of the range.
    __device__ __forceinline__ bool advance(const TreeParams &tp, int per_set) {
        x += chunks + kTreeUnitCost;
        if (x >= end) return false;
        if (++unit == units) {
            unit = 0;
            do {
                ++s;
                enter(tp, per_set);
            } while (units == 0);
        }
        return true;
    }
    // The worker's first segment, in the unit that holds position `start`, or the next; false: it has none.
    __device__ __forceinline__ bool first(const TreeParams &tp, int per_set, bool whole, long long start) {
        if (whole && x < start) {
            if (!advance(tp, per_set)) return false;
        }
        c0 = (int)max(0LL, min((long long)chunks, start - x - kTreeUnitCost));
        c1 = whole ? chunks : (int)max(0LL, min((long long)chunks, end - x - kTreeUnitCost));
        return c1 > c0;
    }
    __device__ __forceinline__ bool next(const TreeParams &tp, int per_set, bool whole) {
        if (!advance(tp, per_set)) return false;
        c0 = 0;
        c1 = whole ? chunks : (int)max(0LL, min((long long)chunks, end - x - kTreeUnitCost));
        return c1 > 0;
    }
    // (one tile's worth of rows holds every tree where units are single tiles: one set)
    __device__ __forceinline__ int head() const { return kPair ? unit / sets : unit; }
    __device__ __forceinline__ int first_draft(int per_set) const { return kPair ? (unit % sets) * per_set : 0; }
};

// Bits e = 0 .. 63: whether a row sees position pos + e. Positions before ctx are context; bit j of the row's
// mask words (word0: the first) is draft j < n = position ctx + j.
__device__ __forceinline__ unsigned long long tree_visible(const int64_t *words, unsigned long long word0, int pos,
                                                           int ctx, int n) {
    const int d = pos - ctx;
    if (d <= -64) return ~0ull;
    const int j0 = max(d, 0);  // first draft wanted
    unsigned long long v = 0;
    if (j0 < n) {
        auto word = [&](int w) {
            return w == 0 ? word0 : (unsigned long long)__ldg(reinterpret_cast<const long long *>(words) + w);
        };
        const int w = j0 >> 6, sh = j0 & 63;
        v = word(w) >> sh;
        if (sh > 0 && (w + 1) * 64 < n) v |= word(w + 1) << (64 - sh);
        if (n - j0 < 64) v &= (1ull << (n - j0)) - 1ull;
    }
    return d < 0 ? (v << -d) | ((1ull << -d) - 1ull) : v;
}

// The same for the 64 score columns of blocks blk .. blk + 3: the sequence's last block was loaded lo rows early, so
// its token t is column lo + t; columns of later blocks hold nothing.
__device__ __forceinline__ unsigned long long tree_columns(unsigned long long visible, int blk, int nblk, int lo) {
    const int last = nblk - 1 - blk;
    if (last >= 4) return visible;
    if (last < 0) return 0ull;
    const unsigned long long before = visible & ((1ull << (16 * last)) - 1ull);
    const unsigned long long tokens = (visible >> (16 * last)) & ((1ull << (kBlock - lo)) - 1ull);
    return before | (tokens << (16 * last + lo));
}

// One warp's copies, issued by its first lane: the K chunks of the worker's range and each unit's Q rows, or the V
// chunks. Lane i < 8 holds the id of a chunk's i-th block, and the next chunk's ahead of use.
template <int D, bool kPair, bool kKeysAndQ>
__device__ __forceinline__ void tree_produce(const CUtensorMap &tm, const CUtensorMap &tmq, const TreeParams &tp,
                                             TreeWalk<D, kPair> at, uint8_t *base, TreeBars &b, int per_set,
                                             int tile_tokens, int q_tokens, bool whole, int lane) {
    using C = TreeCfg<D, kPair>;
    constexpr int NS = C::kStages, CB = C::kChunkBlocks;
    const DecodeParams &p = tp.d;
    uint64_t *full = kKeysAndQ ? b.k_full : b.v_full, *empty = kKeysAndQ ? b.k_empty : b.v_empty;
    uint8_t *ring = base + (kKeysAndQ ? C::kKOff : C::kVOff);
    const uint64_t policy = l2_evict_first();
    bool ok = true;
    int seg = 0, r = 0;  // segments, ring position
    do {
        const int h = at.head();
        const int nblk = (at.len + kBlock - 1) / kBlock, last_valid = at.len - (nblk - 1) * kBlock;
        const int32_t *table = p.block_tables + (size_t)at.s * p.max_blocks_per_seq;
        auto id_of = [&](int j) { return lane < CB && j * CB + lane < nblk ? __ldg(table + j * CB + lane) : -1; };
        int ahead = id_of(at.c0);
        for (int j = at.c0; j < at.c1; ++j, ++r) {
            const int st = r % NS, blk = j * CB + lane;
            const int id = ahead;
            if (j + 1 < at.c1) ahead = id_of(j + 1);
            // this lane's block: its tile (outside the tensor, reading as zeros, past the sequence and for a bad
            // id) and its first slot
            int z = -1;
            const int y = blk == nblk - 1 ? last_valid - kBlock : 0;
            if (lane < CB && blk < nblk) {
                if (id < 0 || id >= p.num_blocks) raise_error(PKV_DEVERR_BLOCK_ID);
                else z = id * p.num_kv_heads + h;
            }
            if (r >= NS && !(ok = warp_wait(&empty[st], (r / NS - 1) & 1))) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kStage);
            uint8_t *dst = ring + st * C::kStage;
#pragma unroll 1
            for (int i = 0; i < CB; ++i) {
                const int zi = __shfl_sync(0xffffffffu, z, i), yi = __shfl_sync(0xffffffffu, y, i);
                if (lane == 0) {
                    if constexpr (kKeysAndQ) {  // [half][128 keys][64]
#pragma unroll
                        for (int u = 0; u < C::kHalves; ++u)
                            tma_load_4d_hint(dst + u * C::kHalfRows, &tm, 0, yi, u, zi, &full[st], policy);
                    } else {                    // [block][half][16 keys][64]
                        tma_load_4d_hint(dst, &tm, 0, yi, 0, zi, &full[st], policy);
                    }
                }
                dst += kKeysAndQ ? kBlock * 128 : C::kBlockBytes;
            }
            if (kKeysAndQ && j == at.c0) {  // behind the first chunk's keys, which need not wait for the last S
                if (seg > 0 && !(ok = warp_wait(&b.q_empty, (seg - 1) & 1))) {
                    ++r;
                    break;
                }
                if (lane == 0) {
                    const int t0 = at.first_draft(per_set);
                    const int tiles = kPair && t0 + tile_tokens < at.n ? 2 : 1;
                    mbar_arrive_expect_tx(&b.q_full, tiles * C::kHalves * 128 * p.group * q_tokens);
#pragma unroll 1
                    for (int t = 0; t < tiles * C::kHalves; ++t)
                        tma_load_4d(base + (t / C::kHalves) * C::kQBytes + (t % C::kHalves) * C::kHalfRows, &tmq, 0,
                                    t % C::kHalves, h * p.group, at.q0 + t0 + (t / C::kHalves) * tile_tokens, &b.q_full);
                }
                ++seg;
            }
        }
    } while (ok && at.next(tp, per_set, whole));
    if (!ok && lane == 0) raise_error(PKV_DEVERR_TIMEOUT);
    // no copy may land after the CTA is gone
    for (int i = max(0, r - NS); i < r; ++i) mbar_wait(&full[i % NS], (i / NS) & 1);
    if (seg > 0) mbar_wait(&b.q_full, (seg - 1) & 1);
}

// Adds what the values cleaner zeroed at positions [from, to) of a sequence to the columns d0 .. d0 + cols - 1 of a
// row that this thread has written (dst, or the state po): an element that meets one is not finite whatever its weight.
// Not in line: it is seldom called, and the epilogue has no registers for it.
__device__ __noinline__ void tree_add_zeroed(const DecodeParams &p, const int64_t *words, int s, int h, int from, int to,
                                             int ctx, int head_dim, int d0, int cols, __nv_bfloat16 *dst, float *po) {
#pragma unroll 1
    for (int ps = from; ps < to; ++ps) {
        if (ps >= ctx && !((__ldg(words + (ps - ctx) / 64) >> ((ps - ctx) % 64)) & 1)) continue;
        const int pb = __ldg(p.block_tables + (size_t)s * p.max_blocks_per_seq + ps / kBlock);
        if (pb < 0 || pb >= p.num_blocks) continue;
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v_cache) +
                                 (((size_t)pb * p.num_kv_heads + h) * kBlock + ps % kBlock) * head_dim + d0;
#pragma unroll 1
        for (int c = 0; c < cols; c += 8) {
            const uint4 w = *reinterpret_cast<const uint4 *>(v + c);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = __uint_as_float(e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
                if (fabsf(x) < INFINITY) continue;
                if (dst) dst[c + e] = __float2bfloat16_rn(__bfloat162float(dst[c + e]) + x);
                else po[c + e] += x;
            }
        }
    }
}

template <int D, bool kPair>
__global__ void __launch_bounds__(TreeCfg<D, kPair>::kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const TreeParams tp, float *partials,
                          TreeCut *cuts, const int tile_tokens, const int q_tokens) {
    using C = TreeCfg<D, kPair>;
    constexpr int NS = C::kStages;
    const DecodeParams &p = tp.d;
    extern __shared__ __align__(1024) uint8_t tree_smem[];  // (three stages leave no room to align it by hand)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = p.group, per_set = C::kTiles * tile_tokens;
    const bool whole = cuts == nullptr;
    uint8_t *const base = tree_smem;
    if (smem_u32(base) & 1023u) {  // the swizzle's atoms would not be where the descriptors say
        if (tid == 0) {
            raise_error(PKV_DEVERR_TIMEOUT);
            if (cuts) cuts[blockIdx.x].segments = 0;  // (the merge reads every CTA's record)
        }
        return;
    }
    TreeBars &b = *reinterpret_cast<TreeBars *>(base + C::kBarOff);
    if (tid == 0) {
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        mbar_init(&b.q_full, 1);
        mbar_init(&b.q_empty, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&b.k_full[i], 1);
            mbar_init(&b.k_empty[i], 1);
            mbar_init(&b.v_full[i], 1);
            mbar_init(&b.v_empty[i], 1);
            mbar_init(&b.v_clean[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.s_full[i], 1);
            mbar_init(&b.p_full[i], 4);
            mbar_init(&b.o_done[i], 1);
            mbar_init(&b.x_full[i], 4);
            mbar_init(&b.x_done[i], 4);
        }
        mbar_init(&b.drain, 1);
        b.any_bad = 0;
        b.start_seq = -1;
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(&b.tmem_base, C::kTmemCols);
        tmem_relinquish();
    }

    // ---- this CTA's range of the line: a scan of the sequences' weights ----
    {
        const int S = p.num_seqs, per = (S + C::kThreads - 1) / C::kThreads;
        const int s_lo = min(S, tid * per), s_hi = min(S, s_lo + per);
        int len, q0, n;
        long long local = 0;
        for (int s = s_lo; s < s_hi; ++s)
            local += TreeWalk<D, kPair>::weigh(tp, s, per_set, blockIdx.x == 0, len, q0, n);
        long long incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) b.warp_sum[warp] = incl;
        __syncthreads();
        long long before = incl - local, total = 0;
        for (int w = 0; w < C::kThreads / 32; ++w) {
            if (w < warp) before += b.warp_sum[w];
            total += b.warp_sum[w];
        }
        const int W = tree_workers(total);
        const long long start = total * blockIdx.x / W;
        if ((int)blockIdx.x < W && start >= before && start < before + local) {
            long long at = before;
            for (int s = s_lo; s < s_hi; ++s) {
                const long long wt = TreeWalk<D, kPair>::weigh(tp, s, per_set, false, len, q0, n);
                if (start < at + wt) {
                    b.start_seq = s;
                    b.start_in = start - at;
                    b.start_rows[0] = len, b.start_rows[1] = q0, b.start_rows[2] = n;
                    break;
                }
                at += wt;
            }
        }
        if (tid == 0) b.total = total;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();  // the merge may be set up; it waits for the states
    const uint32_t tmem = b.tmem_base;
    const long long T = b.total;
    const int W = tree_workers(T), w = blockIdx.x;
    TreeWalk<D, kPair> at;
    bool work = w < W && T > 0;
    if (work) {
        const long long start = T * w / W;
        at.s = b.start_seq;
        at.len = b.start_rows[0], at.q0 = b.start_rows[1], at.n = b.start_rows[2];
        at.derive(tp, per_set);
        at.unit = (int)(b.start_in / (at.chunks + kTreeUnitCost));
        at.x = start - (b.start_in - (long long)at.unit * (at.chunks + kTreeUnitCost));
        at.end = T * (w + 1) / W;
        work = at.first(tp, per_set, whole, start);
    }
    if (!work) {
        if (cuts && tid == 0) cuts[w].segments = 0;
        __syncthreads();
        if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
        return;
    }
    const uint32_t q_s = smem_u32(base), k_s = smem_u32(base + C::kKOff), v_s = smem_u32(base + C::kVOff);

    if (warp < 4) {
        setmaxnreg_dec<C::kLowRegs>();
        if (warp == 0) {
            // ------------------------------ TMA: Q and K ------------------------------
            tree_produce<D, kPair, true>(tmk, tmq, tp, at, base, b, per_set, tile_tokens, q_tokens, whole, lane);
        } else if (warp == 1) {
            // ------------------------------ MMA issuer ------------------------------
            if (lane == 0) {
                constexpr uint32_t idesc_s = idesc_bf16_f32(C::kRows, C::kKeys, false, false);
                constexpr uint32_t idesc_o = idesc_bf16_f32(C::kRows, D, false, true);
                bool ok = true;
                int seg = 0, r0 = 0;
                uint32_t p_parity = 0;  // bit of a side
                auto issue_s = [&](int side, int r) {
                    const uint64_t qd = smem_desc_sw128(q_s + (kPair ? side * C::kQBytes : 0), 16, 1024);
                    const uint64_t kd = smem_desc_sw128(k_s + (r % NS) * C::kStage, 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kHalfRows + (kk & 3) * 32;
                        umma_bf16(tmem + side * C::kSideCols, desc_add(qd, off), desc_add(kd, off), idesc_s, kk > 0);
                    }
                };
                // `first`: O starts here; `split`: the remainders' product too (compiled apart: with a branch
                // between the MMAs 64 trees over 32 q / 8 kv heads took 80 us, 75 us so)
                auto issue_pv = [&](int side, int r, bool first, bool split) {
                    const uint64_t vd0 = smem_desc_sw128(v_s + (r % NS) * C::kStage, kBlock * 128, 1024);
                    const uint32_t d = tmem + side * C::kSideCols + C::kOCol, p0 = tmem + side * C::kSideCols;
#pragma unroll
                    for (int kk = 0; kk < C::kChunkBlocks; ++kk)
                        umma_bf16_tmem_a(d, p0 + (kk >> 1) * 32 + (kk & 1) * 8, desc_add(vd0, kk * C::kBlockBytes),
                                         idesc_o, kk > 0 || !first);
                    if (split) {
#pragma unroll 1
                        for (int kk = 0; kk < C::kChunkBlocks; ++kk)
                            umma_bf16_tmem_a(d, p0 + (kk >> 1) * 32 + (kk & 1) * 8 + 16,
                                             desc_add(vd0, kk * C::kBlockBytes), idesc_o, true);
                    }
                };
                auto wait_k = [&](int r) { return mbar_wait(&b.k_full[r % NS], (r / NS) & 1); };
                do {
                    const int nc = at.c1 - at.c0;
                    const int tiles = kPair && at.first_draft(per_set) + tile_tokens < at.n ? 2 : 1;
                    if (!(ok = mbar_wait(&b.q_full, seg & 1))) break;
                    auto values_ready = [&](int k) {
                        const int st = (r0 + k) % NS;
                        return mbar_wait(&b.v_full[st], ((r0 + k) / NS) & 1) &&
                               mbar_wait(&b.v_clean[st], ((r0 + k) / NS) & 1);
                    };
                    auto weights_ready = [&](int side) {
                        const bool good = mbar_wait(&b.p_full[side], (p_parity >> side) & 1);
                        p_parity ^= 1u << side;
                        tc_fence_after();
                        return good;
                    };
                    if constexpr (kPair) {
                        if (!(ok = wait_k(r0))) break;
                        tc_fence_after();
                        for (int t = 0; t < tiles; ++t) {
                            issue_s(t, r0);
                            umma_commit(&b.s_full[t]);
                        }
                        umma_commit(&b.k_empty[r0 % NS]);
                        for (int k = 0; k < nc && ok; ++k) {
                            ok = values_ready(k) && (k + 1 == nc || wait_k(r0 + k + 1));
                            for (int t = 0; t < tiles && ok; ++t) {
                                if (!(ok = weights_ready(t))) break;
                                issue_pv(t, r0 + k, k == 0, tree_split(at.len - at.n));
                                if (k + 1 < nc) {
                                    issue_s(t, r0 + k + 1);
                                    umma_commit(&b.s_full[t]);
                                } else {
                                    umma_commit(&b.o_done[t]);
                                }
                            }
                            if (!ok) break;
                            umma_commit(&b.v_empty[(r0 + k) % NS]);
                            if (k + 1 < nc) umma_commit(&b.k_empty[(r0 + k + 1) % NS]);
                            if (k + 2 >= nc && k + 1 < nc) umma_commit(&b.q_empty);
                            if (nc == 1) umma_commit(&b.q_empty);
                        }
                    } else {
                        // S of chunk k + 1 goes to the other side before P V of chunk k
                        auto scores = [&](int k) {
                            if (!wait_k(r0 + k)) return false;
                            tc_fence_after();
                            issue_s(k & 1, r0 + k);
                            umma_commit(&b.s_full[k & 1]);
                            umma_commit(&b.k_empty[(r0 + k) % NS]);
                            if (k == nc - 1) umma_commit(&b.q_empty);
                            return true;
                        };
#pragma unroll 1
                        for (int k = -1; k < nc && ok; ++k) {
                            if (k + 1 < nc && !(ok = scores(k + 1))) break;
                            if (k < 0) continue;
                            if (!(ok = values_ready(k) && weights_ready(k & 1))) break;
                            issue_pv(k & 1, r0 + k, k < 2, tree_split(at.len - at.n));
                            umma_commit(&b.v_empty[(r0 + k) % NS]);
                            if (k + 2 >= nc) umma_commit(&b.o_done[k & 1]);
                        }
                    }
                    r0 += nc;
                    ++seg;
                } while (ok && at.next(tp, per_set, whole));
                if (!ok) raise_error(PKV_DEVERR_TIMEOUT);
                umma_commit(&b.drain);  // every MMA has finished before the tensor memory is released
                mbar_wait(&b.drain, 0);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ------------------------------ TMA: V ------------------------------
            tree_produce<D, kPair, false>(tmv, tmq, tp, at, base, b, per_set, tile_tokens, q_tokens, whole, lane);
        } else {
            // ------------------------------ the drafts' values ------------------------------
            bool ok = true;
            int r0 = 0;
            do {
                const int nc = at.c1 - at.c0, first = tree_first_clean(at.len - at.n);
                const int nblk = (at.len + kBlock - 1) / kBlock, lo = nblk * kBlock - at.len;
                // every chunk is waited for and passed on, drafts or not, so that no stage's phase runs
                // away from this role's count
                for (int k = 0; k < nc && ok; ++k) {
                    const int st = (r0 + k) % NS;
                    if (!(ok = warp_wait(&b.v_full[st], ((r0 + k) / NS) & 1))) break;
                    const int blk0 = (at.c0 + k) * C::kChunkBlocks;
                    const int b_lo = max(0, first / kBlock - blk0), b_hi = min(C::kChunkBlocks, nblk - blk0);
                    uint8_t *vst = base + C::kVOff + st * C::kStage;
                    for (int i = b_lo * (C::kBlockBytes / 16) + lane; i < b_hi * (C::kBlockBytes / 16); i += 32) {
                        const uint4 v = reinterpret_cast<const uint4 *>(vst)[i];
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                        uint32_t keep[4];
                        bool bad = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            keep[e] = ((x[e] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) |
                                      ((x[e] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
                            bad |= keep[e] != ~0u;
                        }
                        if (bad) {
                            const int blk = blk0 + i / (C::kBlockBytes / 16), row = (i >> 3) & 15;
                            const int pos = blk * kBlock + row - (blk == nblk - 1 ? lo : 0);
                            if (pos >= first) {
                                reinterpret_cast<uint4 *>(vst)[i] =
                                    make_uint4(x[0] & keep[0], x[1] & keep[1], x[2] & keep[2], x[3] & keep[3]);
                                *reinterpret_cast<volatile int *>(&b.any_bad) = 1;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.v_clean[st]);
                }
                r0 += nc;
            } while (ok && at.next(tp, per_set, whole));
            if (!ok && lane == 0) raise_error(PKV_DEVERR_TIMEOUT);
        }
    } else {
        setmaxnreg_inc<C::kHighRegs>();
        // ------------------------------ softmax ------------------------------
        const int side = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
        const int row_draft = row / g, row_head = row - row_draft * g;
        const uint32_t lane_cols = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t cols = lane_cols + side * C::kSideCols;
        // scores stay raw: x * sl is the log2-domain score, the sign is folded in; a scale of 0 becomes one that
        // leaves every score 0, so that a masked -inf stays -inf
        const float sl = fmaxf(fabsf(p.scale_log2), 1e-30f);
        float2 *xch = reinterpret_cast<float2 *>(base + C::kXchOff);
        bool ok = true;
        int scount = 0, seg = 0;
        uint32_t o_parity = 0;  // bit of a side
        TreeCut cut{0, 0, 0, 0};
        do {
            const int nc = at.c1 - at.c0, h = at.head();
            const int tok0 = at.first_draft(per_set) + (kPair ? side * tile_tokens : 0);
            const int rows = max(0, min(at.n - tok0, tile_tokens)) * g;
            const bool row_ok = row < rows;
            const int draft = tok0 + row_draft;
            const int64_t *words = tp.mask + (size_t)(at.q0 + (row_ok ? draft : 0)) * tp.mask_words;
            const unsigned long long word0 = (unsigned long long)__ldg(reinterpret_cast<const long long *>(words));
            const int ctx = at.len - at.n;
            const int nblk = (at.len + kBlock - 1) / kBlock, lo = nblk * kBlock - at.len;
            const bool warp_rows = quad * 32 < rows;   // a warp without rows only keeps the barriers' count
            float m = -INFINITY, l = 0.f;
            const int k_step = kPair ? 1 : 2, k_first = kPair ? 0 : side;
            const bool active = !kPair || rows > 0;    // (the MMA thread leaves an empty second tile out)
            for (int k = k_first; active && k < nc; k += k_step) {
                if (!(ok = warp_wait(&b.s_full[side], scount++ & 1))) break;
                if (warp_rows) {
                    tc_fence_after();
                    const int j = at.c0 + k;
                    // only chunks that hold drafts or the sequence's end need masks
                    const bool masked = (j + 1) * C::kKeys > ctx || (j + 1) * C::kChunkBlocks >= nblk;
                    // The row of S is read twice, for the max and for the weights, in short rolled loops, and what
                    // only some chunks need stands apart: one warp a scheduler and side runs this code, and
                    // its time follows the instructions that must be fetched (unrolled over the row, with
                    // the masks in line, 5.2 warps waited for an instruction to each one issued; so 0.31).
                    if (__builtin_expect(masked || p.scale_log2 <= 0.f, 0)) {
                        // S rewritten: the sign of the scale folded in, -inf where the row does not see
                        const float f = p.scale_log2 > 0.f ? 1.f : p.scale_log2 < 0.f ? -1.f : 0.f;
                        unsigned long long see[2] = {~0ull, ~0ull};
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int blk = j * C::kChunkBlocks + 4 * i;
                                see[i] = tree_columns(tree_visible(words, word0, blk * kBlock, ctx, at.n), blk, nblk, lo);
                            }
                        }
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t bits = (uint32_t)((q & 2 ? see[1] : see[0]) >> (q & 1 ? 32 : 0));
                            if (!__any_sync(0xffffffffu, bits != ~0u || f != 1.f)) continue;
                            float x[32];
                            tmem_ld32(cols + q * 32, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = bits & (1u << e) ? x[e] * f : -INFINITY;
                            tmem_st32(cols + q * 32, x);
                        }
                        tmem_wait_st();
                    }
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        float x[2][32];
                        tmem_ld32(cols + half * 64, x[0]);
                        tmem_ld32(cols + half * 64 + 32, x[1]);
                        tmem_wait_ld();
                        float mxs[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                mxs[(e >> 1) & 3] = max3f(mxs[(e >> 1) & 3], x[q][e], x[q][e + 1]);
                        mx = fmaxf(max3f(mxs[0], mxs[1], mxs[2]), mxs[3]);
                    }
                    const float m_new = fmaxf(m, mx * sl);
                    const bool move = m_new > m + 8.f;
                    const float m_use = move ? m_new : m;
                    const float ms = m_use == -INFINITY ? 0.f : m_use;
                    const float alpha = ex2_approx(m - ms);
                    // O is quiescent: P V of this side's previous chunk ran before this S
                    if (__builtin_expect(k >= k_step && __any_sync(0xffffffffu, move && m != -INFINITY), 0)) {
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
                    // P over each quarter's score columns: keys 32 q + 2 i, + 1 at column 32 q + i, remainders at + 16
                    const uint64_t sl2 = pack_f2(sl, sl), nms2 = pack_f2(-ms, -ms);
                    uint64_t rss[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) rss[i] = pack_f2(0.f, 0.f);
                    if (__builtin_expect(tree_split(ctx), 0)) {
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            float x[32];
                            uint32_t hi[16], rem[16];
                            tmem_ld32(cols + q * 32, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float a0, a1;
                                unpack_f2(fma_f2(pack_f2(x[2 * i], x[2 * i + 1]), sl2, nms2), a0, a1);
                                const float e0 = ex2_approx(a0), e1 = ex2_approx(a1);
                                rss[i & 3] = add_f2(rss[i & 3], pack_f2(e0, e1));
                                const __nv_bfloat162 ph = __floats2bfloat162_rn(e0, e1);
                                hi[i] = *reinterpret_cast<const uint32_t *>(&ph);
                                const __nv_bfloat162 pl = __floats2bfloat162_rn(e0 - __uint_as_float(hi[i] << 16),
                                                                                e1 - __uint_as_float(hi[i] & 0xffff0000u));
                                rem[i] = *reinterpret_cast<const uint32_t *>(&pl);
                            }
                            tmem_st16(cols + q * 32, hi);
                            tmem_st16(cols + q * 32 + 16, rem);
                        }
                    } else {
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            float x[2][32];
                            tmem_ld32(cols + half * 64, x[0]);
                            tmem_ld32(cols + half * 64 + 32, x[1]);
                            tmem_wait_ld();
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                uint32_t hi[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    float a0, a1;
                                    unpack_f2(fma_f2(pack_f2(x[q][2 * i], x[q][2 * i + 1]), sl2, nms2), a0, a1);
                                    const float e0 = ex2_approx(a0), e1 = ex2_approx(a1);
                                    rss[i & 3] = add_f2(rss[i & 3], pack_f2(e0, e1));
                                    const __nv_bfloat162 ph = __floats2bfloat162_rn(e0, e1);
                                    hi[i] = *reinterpret_cast<const uint32_t *>(&ph);
                                }
                                tmem_st16(cols + half * 64 + q * 32, hi);
                            }
                        }
                    }
                    tmem_wait_st();
                    float rs[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) unpack_f2(rss[i], rs[2 * i], rs[2 * i + 1]);
                    l += ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p_full[side]);
            }
            // ---- the segment ends here ----
            const bool both = nc > 1;                  // (two sides on one tile take its chunks in turn)
            const bool uncut = at.c0 == 0 && at.c1 == at.chunks;
            if (ok) {
                if constexpr (kPair) {
                    if (active) {
                        ok = warp_wait(&b.o_done[side], o_parity & 1);
                        o_parity ^= 1;
                    }
                } else {
                    xch[side * C::kRows + row] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.x_full[side]);
                    ok = warp_wait(&b.x_full[side ^ 1], seg & 1);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (ok && (t == 0 || both)) {
                            ok = warp_wait(&b.o_done[t], (o_parity >> t) & 1);
                            o_parity ^= 1u << t;
                        }
                }
            }
            if (ok && warp_rows) {
                tc_fence_after();
                float f[2] = {1.f, 0.f}, M = m, L = l;
                if constexpr (!kPair) {
                    const float2 other = xch[(side ^ 1) * C::kRows + row];
                    M = fmaxf(m, other.x);
                    const float ms = M == -INFINITY ? 0.f : M;
                    f[side] = ex2_approx(m - ms);
                    f[side ^ 1] = ex2_approx(other.x - ms);
                    L = l * f[side] + other.y * f[side ^ 1];
                }
                const float inv = !uncut ? 1.f : L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;  // (NaN stays)
                f[0] *= inv;
                f[1] *= inv;
                constexpr int kMine = kPair ? D : D / 2;   // columns this side writes
                const int d0 = kPair ? 0 : side * kMine;
                const int unit_row = kPair ? side * C::kRows + row : row;
                float *slot = partials + (size_t)(2 * w + (at.c0 == 0 ? 1 : 0)) * C::kUnitRows * (2 + D);
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                     ((size_t)(at.q0 + (row_ok ? draft : 0)) * p.num_q_heads + h * g + row_head) * D + d0;
                if (!uncut && d0 == 0 && row_ok)
                    *reinterpret_cast<float2 *>(slot + 2 * unit_row) = make_float2(M, L);
                float *po = slot + 2 * C::kUnitRows + (size_t)unit_row * D + d0;
                const uint64_t g0 = pack_f2(f[0], f[0]), g1 = pack_f2(f[1], f[1]), zero = pack_f2(0.f, 0.f);
                const uint32_t col0 = (kPair ? cols : lane_cols) + C::kOCol + d0;
#pragma unroll 1
                for (int c = 0; c < kMine; c += 16) {
                    float o[16], o1[16];
                    tmem_ld16(col0 + c, o);
                    if (!kPair && both) tmem_ld16(col0 + C::kSideCols + c, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        uint64_t v = fma_f2(pack_f2(o[e], o[e + 1]), g0, zero);
                        if (!kPair && both) v = fma_f2(pack_f2(o1[e], o1[e + 1]), g1, v);
                        unpack_f2(v, o[e], o[e + 1]);
                    }
                    if (row_ok && uncut) {
                        uint32_t v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const __nv_bfloat162 v2 = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
                            v[e] = *reinterpret_cast<const uint32_t *>(&v2);
                        }
                        reinterpret_cast<uint4 *>(dst + c)[0] = make_uint4(v[0], v[1], v[2], v[3]);
                        reinterpret_cast<uint4 *>(dst + c)[1] = make_uint4(v[4], v[5], v[6], v[7]);
                    } else if (row_ok) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<float4 *>(po + c + 4 * q) =
                                make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                    }
                }
                if (__builtin_expect(row_ok && *reinterpret_cast<volatile int *>(&b.any_bad) != 0, 0))
                    tree_add_zeroed(p, words, at.s, h, max(tree_first_clean(ctx), at.c0 * C::kKeys),
                                    min(at.len, at.c1 * C::kKeys), ctx, D, d0, kMine, uncut ? dst : nullptr, po);
                tc_fence_before();
            }
            if (!uncut && at.c0 == 0) {  // begun here, ends further on (a worker cuts at most one unit so)
                const long long last = at.x + kTreeUnitCost + at.chunks - 1;  // the unit's last chunk, and its worker
                cut.segments = (int)(((last + 1) * W - 1) / T) - w + 1;
                cut.q_row = at.q0 + at.first_draft(per_set);
                cut.drafts = min(per_set, at.n - at.first_draft(per_set));
                cut.head = h * g;
            }
            if constexpr (!kPair) {
                // the next segment's first P lets the MMA overwrite O: not before both sides have read it
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.x_done[side]);
                if (ok) ok = warp_wait(&b.x_done[side ^ 1], seg & 1);
            }
            ++seg;
        } while (ok && at.next(tp, per_set, whole));
        if (!ok) {
            if (lane == 0) raise_error(PKV_DEVERR_TIMEOUT);
            cut.segments = 0;
        }
        if (cuts && tid == 128) cuts[w] = cut;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Joins the states of every cut unit: a warp per row, four segments' loads in flight.
template <int D>
__global__ void __launch_bounds__(256)
    tree_merge_kernel(__nv_bfloat16 *out, const float *__restrict__ partials, const TreeCut *__restrict__ cuts,
                      int unit_rows, int g, int num_q_heads, int tile_tokens) {
    constexpr int PER = D / 32, NB = 4;
    const int w1 = blockIdx.x, lane = threadIdx.x & 31;
    const int i = blockIdx.y * 8 + (threadIdx.x >> 5);  // (draft, head) of the unit
    pdl_wait();
    const TreeCut cut = cuts[w1];
    if (cut.segments <= 0 || i >= cut.drafts * g) return;
    const int draft = i / g, hg = i - draft * g;
    const int row = (draft / tile_tokens) * 128 + (draft % tile_tokens) * g + hg;
    float M = -INFINITY, L = 0.f, acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < cut.segments; k0 += NB) {
        float m[NB], l[NB], o[NB][PER];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int k = k0 + b;
            m[b] = -INFINITY;
            l[b] = 0.f;
#pragma unroll
            for (int e = 0; e < PER; ++e) o[b][e] = 0.f;
            if (k < cut.segments) {  // the first segment ends its worker's range, the others begin theirs
                const float *slot = partials + (size_t)(2 * (w1 + k) + (k == 0 ? 1 : 0)) * unit_rows * (2 + D);
                m[b] = __ldcg(slot + 2 * row);
                l[b] = __ldcg(slot + 2 * row + 1);
#pragma unroll
                for (int e = 0; e < PER; ++e) o[b][e] = __ldcg(slot + 2 * unit_rows + (size_t)row * D + lane + 32 * e);
            }
        }
        float top = M;
#pragma unroll
        for (int b = 0; b < NB; ++b) top = fmaxf(top, m[b]);
        const float ms = top == -INFINITY ? 0.f : top;  // (rows that have seen nothing yet)
        const float al = ex2_approx(M - ms);
        M = top;
        L *= al;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] *= al;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float f = ex2_approx(m[b] - ms);
            L = fmaf(l[b], f, L);
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(o[b][e], f, acc[e]);
        }
    }
    const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;
    __nv_bfloat16 *dst = out + ((size_t)(cut.q_row + draft) * num_q_heads + cut.head + hg) * D;
#pragma unroll
    for (int e = 0; e < PER; ++e) dst[lane + 32 * e] = __float2bfloat16_rn(acc[e] * inv);
}

// =====================================================================================
// The accepted path: one CTA per (kv heads, layer, sequence). Its first threads look up where each accepted row
// lies and goes; then all rows of K and V are read into shared memory, and written. A step's few rows per
// sequence and layer leave it bound by the chain of lookups, so a CTA takes as many heads as shared memory
// holds (64 sequences, 32 layers, 8 heads, 3.5 rows: 19.1 us with one head a CTA, 13.1 us so).
// =====================================================================================
struct AcceptParams {
    void *const *k_caches, *const *v_caches;
    const int32_t *block_tables, *context_lens, *query_start, *accepted, *num_accepted;
    int32_t *new_lens;
    int max_accepted, num_kv_heads, max_blocks_per_seq, num_blocks;
    int row_vecs;  // 16-byte vectors of a row
    int heads;     // kv heads of a CTA
};

__global__ void __launch_bounds__(128) kv_accept_kernel(const AcceptParams p) {
    extern __shared__ __align__(16) uint4 accept_rows[];  // [K / V][accepted][heads][row_vecs]
    __shared__ int from_s[PKV_MAX_ACCEPTED], to_s[PKV_MAX_ACCEPTED];  // slots (block * 16 + offset); from < 0: no move
    const int h0 = blockIdx.x * p.heads, layer = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
    const bool lead = blockIdx.x == 0 && layer == 0;
    const int len = __ldg(p.context_lens + s), cap = p.max_blocks_per_seq * kBlock;
    const long long n = (long long)__ldg(p.query_start + s + 1) - __ldg(p.query_start + s);
    int a = __ldg(p.num_accepted + s);
    if (len < 0 || len > cap || n < 0 || n > len) {
        if (lead && tid == 0) {
            raise_error(PKV_DEVERR_LENGTH);
            p.new_lens[s] = len;
        }
        return;
    }
    const int base = len - (int)n, most = min((int)n, p.max_accepted);
    if (a < 0 || a > most) {
        if (lead && tid == 0) raise_error(PKV_DEVERR_LENGTH);
        a = a < 0 ? 0 : most;
    }
    if (lead && tid == 0) p.new_lens[s] = base + a;
    uint4 *kc = static_cast<uint4 *>(p.k_caches[layer]), *vc = static_cast<uint4 *>(p.v_caches[layer]);
    if (((reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) & 15) != 0 || !kc || !vc) {
        if (tid == 0 && blockIdx.x == 0 && s == 0) raise_error(PKV_DEVERR_POINTER);
        return;
    }
    if (tid < a) {
        const int32_t *table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
        const int d = __ldg(p.accepted + (size_t)s * p.max_accepted + tid);
        int from = -1, to = -1;
        if (d < 0 || d >= n) {
            if (lead) raise_error(PKV_DEVERR_INDEX);
        } else if (d != tid) {
            const int fb = __ldg(table + (base + d) / kBlock), tb = __ldg(table + (base + tid) / kBlock);
            if (fb < 0 || fb >= p.num_blocks || tb < 0 || tb >= p.num_blocks) {
                if (lead) raise_error(PKV_DEVERR_BLOCK_ID);
            } else {
                from = fb * kBlock + (base + d) % kBlock;
                to = tb * kBlock + (base + tid) % kBlock;
            }
        }
        from_s[tid] = from;
        to_s[tid] = to;
    }
    __syncthreads();
    const int heads = min(p.heads, p.num_kv_heads - h0), per_row = heads * p.row_vecs, total = 2 * a * per_row;
    auto each = [&](auto move) {
        for (int i = tid; i < total; i += blockDim.x) {
            const int r = i / per_row, j = r >> 1, in_row = i - r * per_row;
            if (from_s[j] < 0) continue;
            const int h = in_row / p.row_vecs, c = in_row - h * p.row_vecs;
            auto at = [&](int slot) {
                return (((size_t)(slot >> 4) * p.num_kv_heads + h0 + h) * kBlock + (slot & 15)) * p.row_vecs + c;
            };
            move(i, (r & 1) ? vc : kc, at(from_s[j]), at(to_s[j]));
        }
    };
    each([&](int i, const uint4 *cache, size_t from, size_t) { accept_rows[i] = cache[from]; });
    __syncthreads();
    each([&](int i, uint4 *cache, size_t, size_t to) { cache[to] = accept_rows[i]; });
}

}  // namespace pkv
