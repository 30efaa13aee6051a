// pkv_verify.cuh -- which drafted tokens stand: the walk down a tree of drafts
// against the target's probabilities, and the token that follows it, from
// random numbers that the caller gives.
#pragma once

#include <cooperative_groups.h>

#include "pkv_kernels.cuh"

namespace pkv {

struct VerifyParams {
    int32_t *accepted, *num_accepted;   // [num_seqs][max_accepted], [num_seqs]
    int64_t *next_tokens;               // [num_seqs]
    const int64_t *tokens;              // [num_queries]
    const int32_t *parents, *query_start;
    const void *target, *draft;         // [num_queries][vocab], rows target_stride, draft_stride apart; draft may be null
    int64_t target_stride, draft_stride;
    const float *uniforms, *final_uniforms;
    int num_queries, max_query_len, max_accepted, vocab;
    int vector_rows;                    // every row starts on 16 bytes
};

// =====================================================================================
// A cluster of CTAs takes a sequence. Every draft's parent, token, random number and the two probabilities of
// its token are gathered at once into shared memory, and every CTA of the cluster walks the tree by itself:
//   at a node, with p and q the target's and the draft model's probabilities behind it, the children are tried in
//   order; what may still be drawn is r = max(p - A q, 0) with sum Z, at first A = 0 and, by definition, Z = 1;
//   a child with token x stands if u q(x) Z < r(x); else A grows by Z and Z becomes the new sum.
// (After k refusals of samples of q the remaining distribution is max(r_k / Z_k - q, 0) normalised; as each step takes off
// a multiple of the same q, r_k+1 = max(r_k - Z_k q, 0) = max(p - A_k+1 q, 0), so no step needs the one before it.)
// Without q a draft is certain: q(x) = 1, and a refused token leaves r. Where the walk ends, the first token whose
// running sum of r exceeds u Z follows.
//
// Only a refusal and the end of the walk read rows of the vocabulary, once each: the CTAs take a stretch each, the warps a
// stretch of that, and the CTAs' sums go to all of the cluster through distributed shared memory. The warps'
// sums of the last pass are kept, so the token is looked for in one warp's stretch only.
//
// Probabilities become multiples of 2^-60 in 64 bits, and sums of them are exact whatever their order: the place
// where a running sum passes u Z must not move, for among 10^5 borders sums in 32 bits would move one past u Z in one
// call of some hundred. (Sums in fp64 would do too, but this card does two such operations a clock and SM.)
// =====================================================================================
constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxRows = PKV_TREE_MAX_DRAFTS;
using Fixed = unsigned long long;

// A probability in units of 2^-60, truncated. Negative numbers and NaN count as 0, more than 2 as 2.
__device__ __forceinline__ Fixed to_fixed(float x) { return __float2ull_rz(fminf(fmaxf(x, 0.f), 2.f) * 0x1p60f); }

// A: units of 2^-50, which leave room for the sums of 1024 refusals.
constexpr Fixed kVerifyOne = 1ull << 50;

// max(p - A q, 0)
__device__ __forceinline__ Fixed residual(Fixed p, Fixed q, Fixed a) {
    if (a == kVerifyOne) return p > q ? p - q : 0;
    const Fixed hi = __umul64hi(a, q), aq = (hi << 14) | ((a * q) >> 50);
    return hi >> 49 == 0 && p > aq ? p - aq : 0;
}

template <typename T>
__device__ __forceinline__ float prob(const T *row, int64_t i) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(row[i]);
    else return row[i];
}

// E elements of a row from v on, zeros past the vocabulary.
template <typename T, int E>
__device__ __forceinline__ void load_probs(const T *row, int v, int vocab, bool vec, float (&x)[E]) {
    if (vec && v + E <= vocab) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(row + v));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[e] = E == 4 ? __uint_as_float(u[e]) : __uint_as_float(e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = v + e < vocab ? prob(row, v + e) : 0.f;
    }
}

__device__ __forceinline__ Fixed warp_sum(Fixed x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One warp's sum of r over [lo, hi), lo a multiple of a step's elements (32 E). a: 0 for r = p.
template <typename T, int E>
__device__ __forceinline__ Fixed sum_residual(const T *p, const T *q, Fixed a, int lo, int hi, int vocab, bool vec,
                                              int lane) {
    constexpr int kStep = 32 * E, kUnroll = 4;
    Fixed sum = 0;
    for (int v0 = lo + lane * E; v0 < hi; v0 += kStep * kUnroll) {
        float x[kUnroll][E], y[kUnroll][E];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int v = v0 + k * kStep;
            load_probs<T, E>(p, v < hi ? v : vocab, vocab, vec, x[k]);
            if (a) load_probs<T, E>(q, v < hi ? v : vocab, vocab, vec, y[k]);
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const Fixed f = to_fixed(x[k][e]);
                sum += a ? residual(f, to_fixed(y[k][e]), a) : f;
            }
    }
    return warp_sum(sum);
}

struct VerifyShared {
    int parent[kVerifyMaxRows];          // -1: never tried
    int token[kVerifyMaxRows];           // -1: outside the vocabulary
    float p[kVerifyMaxRows], q[kVerifyMaxRows], u[kVerifyMaxRows];  // of the draft's token, behind its parent
    int path[kVerifyMaxRows];
    int refused[kVerifyMaxRows];         // without q: rows of the refused tokens, each token once
    Fixed cta_sum[2][16];                // by pass and CTA of the cluster
    Fixed warp_sums[kVerifyWarps], fine[kVerifyWarps];
};

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_drafts_kernel(const VerifyParams a) {
    namespace cg = cooperative_groups;
    constexpr int E = 16 / sizeof(T), kStep = 32 * E;
    extern __shared__ __align__(16) unsigned char verify_smem[];
    VerifyShared &sh = *reinterpret_cast<VerifyShared *>(verify_smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int s = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool lead = rank == 0;
    if (lead && tid == 0) a.next_tokens[s] = -1;  // (before the first pass, so before the token that follows)
    const int q0 = __ldg(a.query_start + s);
    const long long nn = (long long)__ldg(a.query_start + s + 1) - q0;
    int32_t *path_out = a.accepted + (size_t)s * a.max_accepted;
    if (nn <= 0 || nn > a.max_query_len || q0 < 0 || q0 + nn > a.num_queries) {  // (the whole cluster)
        if (lead) {
            if (tid == 0) {
                if (nn != 0) raise_error(PKV_DEVERR_LENGTH);
                a.num_accepted[s] = 0;
            }
            for (int i = tid; i < a.max_accepted; i += kVerifyThreads) path_out[i] = -1;
        }
        return;
    }
    const int n = (int)nn, V = a.vocab;
    const T *target = static_cast<const T *>(a.target) + (size_t)q0 * a.target_stride;
    const T *draft = a.draft ? static_cast<const T *>(a.draft) + (size_t)q0 * a.draft_stride : nullptr;
    const bool vec = a.vector_rows != 0;

    for (int i = tid; i < n; i += kVerifyThreads) {
        int up = i == 0 ? -1 : __ldg(a.parents + q0 + i);
        const int64_t x = i == 0 ? -1 : __ldg(reinterpret_cast<const long long *>(a.tokens) + q0 + i);
        float px = 0.f, qx = 1.f;
        if (i > 0) {
            const bool known = x >= 0 && x < V;
            if (up < 0 || up >= i || !known) {
                if (lead) raise_error(PKV_DEVERR_INDEX);
                if (up < 0 || up >= i) up = -1;
            }
            if (up >= 0 && known) {
                px = prob(target + (size_t)up * a.target_stride, x);
                if (draft) qx = prob(draft + (size_t)up * a.draft_stride, x);
            }
            sh.token[i] = known ? (int)x : -1;
            sh.u[i] = __ldg(a.uniforms + q0 + i);
        }
        sh.parent[i] = up;
        sh.p[i] = px;
        sh.q[i] = qx;
    }
    __syncthreads();

    // the vocabulary's stretch of a CTA, of a warp, and of a warp of those that look into one warp's stretch
    const int per_warp = (V + ctas * kVerifyWarps * kStep - 1) / (ctas * kVerifyWarps * kStep) * kStep;
    const int per_fine = (per_warp + kVerifyWarps * kStep - 1) / (kVerifyWarps * kStep) * kStep;
    const int my_lo = (int)min((long long)V, (long long)(rank * kVerifyWarps + warp) * per_warp);
    const int my_hi = (int)min((long long)V, (long long)my_lo + per_warp);

    int passes = 0;
    // The sum of r over the vocabulary (that of p where A is 0), left by warp and by CTA too.
    auto pass = [&](int node, Fixed A) -> Fixed {
        const Fixed mine = sum_residual<T, E>(target + (size_t)node * a.target_stride,
                                              draft ? draft + (size_t)node * a.draft_stride : nullptr, A, my_lo, my_hi,
                                              V, vec, lane);
        __syncthreads();  // (the last pass's sums have been read)
        if (lane == 0) sh.warp_sums[warp] = mine;
        __syncthreads();
        const int slot = passes++ & 1;
        if (warp == 0 && lane < ctas) {
            Fixed sum = 0;
            for (int w = 0; w < kVerifyWarps; ++w) sum += sh.warp_sums[w];
            cluster.map_shared_rank(&sh, lane)->cta_sum[slot][rank] = sum;
        }
        cluster.sync();
        Fixed total = 0;
        for (int c = 0; c < ctas; ++c) total += sh.cta_sum[slot][c];
        return total;
    };

    // ---- the walk: every thread of the cluster keeps the same state ----
    int node = 0, count = 1, refusals = 0, listed = 0;
    Fixed A = 0, Z = 0;     // Z: the sum of r, known once `summed`
    bool summed = false, spent = false;
    if (tid == 0) sh.path[0] = 0;
    // without q: whether the token of draft i has been refused
    auto gone = [&](int i) -> bool {
        bool hit = false;
        for (int j = lane; j < listed; j += 32) hit |= sh.token[sh.refused[j]] == sh.token[i];
        return __any_sync(0xffffffffu, hit);
    };
    for (int from = 1; from < n && count < a.max_accepted;) {
        // the next child of the node
        const bool child = from + lane < n && sh.parent[from + lane] == node;
        const unsigned ballot = __ballot_sync(0xffffffffu, child);
        if (ballot == 0) {
            from += 32;
            continue;
        }
        const int i = from + __ffs(ballot) - 1;
        from = i + 1;
        // u q Z < r: the product of two fp32 numbers is exact in fp64, and where r is p it is taken as it came
        const bool whole = draft ? A == 0 : !gone(i);
        const Fixed have = draft && A ? residual(to_fixed(sh.p[i]), to_fixed(sh.q[i]), A) : whole ? to_fixed(sh.p[i]) : 0;
        const double bar = (double)sh.u[i] * (double)sh.q[i] * (refusals ? (double)Z * 0x1p-60 : 1.0);
        if (bar < (whole ? (double)sh.p[i] : (double)have * 0x1p-60)) {
            node = i;
            if (tid == 0) sh.path[count] = i;
            ++count;
            refusals = listed = 0;
            A = Z = 0;
            summed = spent = false;
            continue;
        }
        if (spent) continue;  // (p and q are the same to the last bit: r stays what it was)
        if (draft) {
            const Fixed A1 = refusals ? A + (Z >> 10) : kVerifyOne;
            const Fixed Z1 = pass(node, A1);
            if (Z1 == 0) {
                spent = true;
                summed = false;   // (the warps' sums are those of nothing)
            } else {
                A = A1;
                Z = Z1;
                summed = true;
                ++refusals;
            }
        } else {
            if (!summed) {
                Z = pass(node, 0);
                summed = true;
            }
            if (Z > have) {
                Z -= have;
                ++refusals;
                if (have) {
                    __syncthreads();
                    if (tid == 0) sh.refused[listed] = i;
                    ++listed;
                    __syncthreads();
                }
            }
        }
    }
    if (!summed) Z = pass(node, A);

    // ---- the token that follows ----
    __syncthreads();
    if (lead) {
        for (int i = tid; i < a.max_accepted; i += kVerifyThreads) path_out[i] = i < count ? sh.path[i] : -1;
        if (tid == 0) a.num_accepted[s] = count;
    }
    if (Z == 0) return;  // a row without a positive probability
    const T *prow = target + (size_t)node * a.target_stride;
    const T *qrow = draft ? draft + (size_t)node * a.draft_stride : nullptr;
    const float u = fminf(fmaxf(__ldg(a.final_uniforms + s), 0.f), 0x1.fffffep-1f);
    const Fixed goal = min((Fixed)__double2ull_rd((double)u * (double)Z), Z - 1);
    // what the refused tokens (without q) take off a stretch's sum
    auto refused_in = [&](int lo, int hi) -> Fixed {
        if (listed == 0) return 0;
        Fixed off = 0;
        for (int j = lane; j < listed; j += 32) {
            const int i = sh.refused[j];
            if (sh.token[i] >= lo && sh.token[i] < hi) off += to_fixed(sh.p[i]);
        }
        return warp_sum(off);
    };
    // the CTA's stretch
    Fixed below = 0, mine = 0;
    for (int c = 0; c <= rank; ++c) {
        const int lo = (int)min((long long)V, (long long)c * kVerifyWarps * per_warp);
        const int hi = (int)min((long long)V, (long long)(c + 1) * kVerifyWarps * per_warp);
        below += mine;
        mine = sh.cta_sum[(passes - 1) & 1][c] - refused_in(lo, hi);
    }
    if (goal < below || goal >= below + mine) return;
    // the warp's stretch
    int w = -1;
    Fixed in_warp = 0;
    do {
        below += in_warp;
        ++w;
        const int lo = (int)min((long long)V, (long long)(rank * kVerifyWarps + w) * per_warp);
        in_warp = sh.warp_sums[w] - refused_in(lo, (int)min((long long)V, (long long)lo + per_warp));
    } while (w < kVerifyWarps - 1 && goal >= below + in_warp);
    const int w_lo = (rank * kVerifyWarps + w) * per_warp, w_hi = (int)min((long long)V, (long long)w_lo + per_warp);
    // the part of it, one to a warp
    const int f_lo = min(w_hi, w_lo + warp * per_fine), f_hi = min(w_hi, f_lo + per_fine);
    const Fixed part = sum_residual<T, E>(prow, qrow, A, f_lo, f_hi, V, vec, lane) - refused_in(f_lo, f_hi);
    if (lane == 0) sh.fine[warp] = part;
    __syncthreads();
    for (int f = 0; f < warp; ++f) below += sh.fine[f];
    if (goal < below || goal >= below + part) return;
    // its step and lane
    for (int v0 = f_lo; v0 < f_hi; v0 += kStep) {
        const int v = v0 + lane * E;
        float x[E], y[E];
        Fixed r[E], sum = 0;
        load_probs<T, E>(prow, v < f_hi ? v : V, V, vec, x);
        if (A) load_probs<T, E>(qrow, v < f_hi ? v : V, V, vec, y);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            r[e] = to_fixed(x[e]);
            if (A) r[e] = residual(r[e], to_fixed(y[e]), A);
            for (int j = 0; j < listed; ++j)
                if (sh.token[sh.refused[j]] == v + e) r[e] = 0;
            sum += r[e];
        }
        Fixed upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Fixed t = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += t;
        }
        const Fixed all = __shfl_sync(0xffffffffu, upto, 31);
        if (goal < below + all) {
            Fixed at = below + upto - sum;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (goal >= at && goal < at + r[e]) a.next_tokens[s] = v + e;
                at += r[e];
            }
            return;
        }
        below += all;
    }
}

}  // namespace pkv
