// pkv_tree.cuh -- drafted tokens: the mask of a tree from its parents,
// attention of a tree's rows over the paged cache, and the move of the
// accepted path's keys and values to consecutive positions.
#pragma once

#include "pkv_kernels.cuh"

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
// the walk meets falling indexes and fills the row's words from the last to the first.
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
// Attention, one warp per (row, query head): 32 tokens at a time, a lane scores one of them.
// =====================================================================================
template <int D>
__global__ void __launch_bounds__(128) tree_attention_kernel(const TreeParams tp) {
    constexpr int PER = D / 32;
    const DecodeParams &p = tp.d;
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.y;
    const int len = seq_len(p, s, blockIdx.x == 0 && threadIdx.x == 0);
    int q0, n;
    if (!tree_rows(tp.query_start, s, len, tp.max_query_len, tp.num_queries, q0, n)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(PKV_DEVERR_LENGTH);
        return;
    }
    const int item = blockIdx.x * 4 + warp;
    const int i = item / p.num_q_heads, hq = item - i * p.num_q_heads;
    if (i >= n) return;
    const int h = hq / p.group;
    const size_t row = (size_t)(q0 + i) * p.num_q_heads + hq;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + row * D;
    for (int d = lane; d < D; d += 32) qs[warp][d] = __bfloat162float(q[d]) * p.scale_log2;
    __syncwarp();
    const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(p.k_cache);
    const __nv_bfloat16 *vc = static_cast<const __nv_bfloat16 *>(p.v_cache);
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    const int64_t *words = tp.mask + (size_t)(q0 + i) * tp.mask_words;
    const int base = len - n;
    float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int t0 = 0; t0 < len; t0 += 32) {
        const int t = t0 + lane, j = t - base;
        const bool see = t < len && (j < 0 || ((__ldg(words + j / 64) >> (j % 64)) & 1) != 0);
        int pb = -1;
        if (see) {
            pb = __ldg(table + t / kBlock);
            if (pb < 0 || pb >= p.num_blocks) {
                raise_error(PKV_DEVERR_BLOCK_ID);
                pb = -1;
            }
        }
        float x = see ? 0.f : -INFINITY;
        if (pb >= 0) {
            const __nv_bfloat16 *kr = kc + (((size_t)pb * p.num_kv_heads + h) * kBlock + (t & 15)) * D;
            for (int d = 0; d < D; ++d) x = fmaf(__bfloat162float(kr[d]), qs[warp][d], x);
        }
        float mx = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
        const float al = exp2f(m - ms), w = exp2f(x - ms);
        m = mn;
        l = l * al + w;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] *= al;
        for (int u = 0; u < min(32, len - t0); ++u) {
            const int b = __shfl_sync(0xffffffffu, pb, u);
            const float wu = __shfl_sync(0xffffffffu, w, u);
            if (b < 0) continue;
            const __nv_bfloat16 *vr = vc + (((size_t)b * p.num_kv_heads + h) * kBlock + ((t0 + u) & 15)) * D;
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(__bfloat162float(vr[lane + 32 * e]), wu, acc[e]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + row * D;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) out[lane + 32 * e] = __float2bfloat16_rn(acc[e] * inv);
}

// =====================================================================================
// The accepted path: one CTA per (kv head, layer, sequence) reads all its rows of K and V into
// shared memory, then writes them.
// =====================================================================================
struct AcceptParams {
    void *const *k_caches, *const *v_caches;
    const int32_t *block_tables, *context_lens, *query_start, *accepted, *num_accepted;
    int32_t *new_lens;
    int max_accepted, num_kv_heads, max_blocks_per_seq, num_blocks;
    int row_vecs;  // 16-byte vectors of a row
};

__global__ void __launch_bounds__(128) kv_accept_kernel(const AcceptParams p) {
    extern __shared__ uint4 rows_s[];  // [2][accepted][row_vecs]
    const int h = blockIdx.x, layer = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
    const bool lead = h == 0 && layer == 0 && tid == 0;
    int len = __ldg(p.context_lens + s);
    const int cap = p.max_blocks_per_seq * kBlock;
    int n = __ldg(p.query_start + s + 1) - __ldg(p.query_start + s);
    bool bad = len < 0 || len > cap || n < 0 || n > len;
    if (bad) {
        if (lead) {
            raise_error(PKV_DEVERR_LENGTH);
            p.new_lens[s] = len;
        }
        return;
    }
    const int base = len - n;
    int a = __ldg(p.num_accepted + s);
    if (a < 0 || a > min(n, p.max_accepted)) {
        if (lead) raise_error(PKV_DEVERR_LENGTH);
        a = a < 0 ? 0 : min(n, p.max_accepted);
    }
    if (lead) p.new_lens[s] = base + a;
    uint4 *kc = static_cast<uint4 *>(p.k_caches[layer]), *vc = static_cast<uint4 *>(p.v_caches[layer]);
    if (((reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) & 15) != 0 || !kc || !vc) {
        if (tid == 0 && h == 0 && s == 0) raise_error(PKV_DEVERR_POINTER);
        return;
    }
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    // the row's first vector in a cache, or -1
    auto at = [&](int pos) -> int64_t {
        const int b = __ldg(table + pos / kBlock);
        if (b < 0 || b >= p.num_blocks) {
            if (layer == 0 && h == 0) raise_error(PKV_DEVERR_BLOCK_ID);
            return -1;
        }
        return (((int64_t)b * p.num_kv_heads + h) * kBlock + pos % kBlock) * p.row_vecs;
    };
    auto each = [&](bool store) {
        for (int idx = tid; idx < 2 * a * p.row_vecs; idx += blockDim.x) {
            const int c = idx % p.row_vecs, r = idx / p.row_vecs;
            const int j = r >> 1;
            uint4 *cache = (r & 1) ? vc : kc;
            const int d = __ldg(p.accepted + (size_t)s * p.max_accepted + j);
            if (d < 0 || d >= n) {
                if (layer == 0 && h == 0 && !store) raise_error(PKV_DEVERR_INDEX);
                continue;
            }
            if (d == j) continue;
            const int64_t from = at(base + d), to = at(base + j);
            if (from < 0 || to < 0) continue;
            if (store) cache[to + c] = rows_s[idx];
            else rows_s[idx] = cache[from + c];
        }
    };
    each(false);
    __syncthreads();
    each(true);
}

}  // namespace pkv
