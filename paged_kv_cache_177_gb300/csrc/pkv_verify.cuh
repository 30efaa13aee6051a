// pkv_verify.cuh -- which drafted tokens stand: the walk down a tree of drafts
// against the target's probabilities, and the token that follows it, from
// random numbers that the caller gives.
#pragma once

#include <cooperative_groups.h>

#include "pkv_prefill_tc.cuh"

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
// A probability becomes a multiple of 2^-44, rounded to nearest, and sums of them are exact whatever their order: the
// place where a running sum passes u Z must not move, for among 10^5 borders sums in 32 bits would move one past u Z in
// one call of some hundred. (The roundings of 10^5 terms move a border by 10^-11, and one past u Z in a call of 10^6.)
// fp64 would do too, but this card adds two of them a clock and SM, and converts fp32 to 64-bit integers as
// slowly: with that 256 rows of 131072 took 93 us.
// =====================================================================================
constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyBlocks = 2;  // of an SM, whose loads overlap: 64 registers a thread
constexpr int kVerifyMaxRows = PKV_TREE_MAX_DRAFTS;
using Fixed = long long;

// x in [0, 1] is cut into a multiple of 2^-22 and the rest's of 2^-44 by adding numbers whose last bit is that:
// the sums' bits, less those of the numbers, are the two integers.
constexpr float kCut1 = 3.f, kCut2 = 0x1.8p-21f;
constexpr uint32_t kCut1Bits = 0x40400000u, kCut2Bits = 0x35400000u;

__device__ __forceinline__ void cut(float x, uint32_t &a, uint32_t &b) {
    const float t = x + kCut1, r = x - (t - kCut1);
    a = __float_as_uint(t);
    b = __float_as_uint(r + kCut2);
}

__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, 0.f), 1.f); }  // (NaN: 0)

__device__ __forceinline__ Fixed to_fixed(float x) {
    uint32_t a, b;
    cut(clean(x), a, b);
    return ((Fixed)(int)(a - kCut1Bits) << 22) + (int)(b - kCut2Bits);
}

// A number of at least 1 as hi + lo, from units of 2^-44. hi = 0: nothing is taken off.
struct Multiple {
    float hi, lo;
};

__device__ __forceinline__ Multiple to_multiple(Fixed a) {
    const float hi = (float)a;
    return {hi * 0x1p-44f, (float)(a - (Fixed)hi) * 0x1p-44f};
}

// u q Z < r for fp32 u and q, Z and r in units of 2^-44: the product of three as the sum of two fp32 numbers, 2^-46 of it
// off. (In fp64, which every warp would pay 16 clocks an operation for, a draft's test took 0.8 us.)
__device__ __forceinline__ bool below(float u, float q, Fixed Z, Fixed r) {
    const Multiple z = to_multiple(Z), a = to_multiple(r);
    const float x = __fmul_rn(u, q), e = fmaf(u, q, -x);
    const float h = __fmul_rn(x, z.hi), l = fmaf(x, z.hi, -h) + fmaf(x, z.lo, e * z.hi);
    return (h - a.hi) + (l - a.lo) < 0.f;
}

// u q < p, exactly: x = u q rounded lies on p's side of the product, or on p.
__device__ __forceinline__ bool below(float u, float q, float p) {
    const float x = u * q;
    return x == p ? fmaf(u, q, -x) < 0.f : x < p;
}

// A q as the sum of two fp32 numbers, 2^-48 of it off; whether p exceeds it by a unit or more. (p, x and y are each
// rounded to units, so what exceeds by less could come out as -1, and with it a whole sum. x is the rounded
// product, which must not be fused into the difference.)
__device__ __forceinline__ bool exceeds(float p, float q, Multiple A, float &x, float &y) {
    x = __fmul_rn(A.hi, q);
    y = fmaf(A.lo, q, fmaf(A.hi, q, -x));
    return (p - x) - y >= 0x1p-44f;
}

// max(p - A q, 0), less than a unit of it as 0: never negative.
__device__ __forceinline__ Fixed residual(float p, float q, Multiple A) {
    p = clean(p);
    q = clean(q);
    if (A.hi == 0.f) return to_fixed(p);
    if (A.hi == 1.f && A.lo == 0.f) return to_fixed(p) - to_fixed(fminf(p, q));
    float x, y;
    if (!exceeds(p, q, A, x, y)) return 0;
    return to_fixed(p) - to_fixed(x) - (int)(__float_as_uint(y + kCut2) - kCut2Bits);
}

template <typename T>
__device__ __forceinline__ float prob(const T *row, int64_t i) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(row[i]);
    else return row[i];
}

// E elements of a row from 16 bytes, and from anywhere, zeros past the vocabulary.
template <typename T, int E>
__device__ __forceinline__ void unpack_probs(const uint4 w, float (&x)[E]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < E; ++e)
        x[e] = E == 4 ? __uint_as_float(u[e]) : __uint_as_float(e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
}

template <typename T, int E>
__device__ __forceinline__ void load_probs(const T *row, int v, int vocab, float (&x)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = v + e < vocab ? prob(row, v + e) : 0.f;
}

__device__ __forceinline__ Fixed warp_sum(Fixed x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One warp's sum of r over [lo, hi), lo a multiple of a step's elements (32 E). Rounds of whole steps of aligned rows are
// loaded ahead of their use, without a branch between the loads (with one between them 64 trees took 55 us, 47 so).
template <typename T, int E>
__device__ __forceinline__ Fixed sum_residual(const T *p, const T *q, Multiple A, int lo, int hi, int vocab, bool vec,
                                              int lane) {
    constexpr int kStep = 32 * E;
    Fixed sum = 0;
    // the cuts of a round's elements are summed in 32 bits: at most 32 numbers of 22 bits
    uint32_t a = 0, b = 0;
    auto each = [&](auto with_q, auto add, auto flush) {
        constexpr bool kQ = decltype(with_q)::value;
        constexpr int kUnroll = (kQ ? 16 : 32) / E;  // 32 registers of loads in flight
        int v0 = lo;
        if (vec) {
            for (; v0 + kStep * kUnroll <= hi; v0 += kStep * kUnroll) {
                uint4 x[kUnroll], y[kUnroll];
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    x[k] = __ldg(reinterpret_cast<const uint4 *>(p + v0 + k * kStep) + lane);
                    if constexpr (kQ) y[k] = __ldg(reinterpret_cast<const uint4 *>(q + v0 + k * kStep) + lane);
                }
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    float xf[E], yf[E];
                    unpack_probs<T, E>(x[k], xf);
                    if constexpr (kQ) unpack_probs<T, E>(y[k], yf);
#pragma unroll
                    for (int e = 0; e < E; ++e) add(clean(xf[e]), kQ ? yf[e] : 0.f);
                }
                flush(kUnroll * E);
            }
        }
        for (; v0 < hi; v0 += kStep) {
            float xf[E], yf[E];
            load_probs<T, E>(p, v0 + lane * E, vocab, xf);
            if constexpr (kQ) load_probs<T, E>(q, v0 + lane * E, vocab, yf);
#pragma unroll
            for (int e = 0; e < E; ++e) add(clean(xf[e]), kQ ? yf[e] : 0.f);
            flush(E);
        }
    };
    if (A.hi == 0.f) {
        each(BoolConst<false>{}, [&](float x, float) {
            uint32_t xa, xb;
            cut(x, xa, xb);
            a += xa;
            b += xb;
        }, [&](uint32_t n) {
            sum += ((Fixed)(int)(a - n * kCut1Bits) << 22) + (int)(b - n * kCut2Bits);
            a = b = 0;
        });
    } else if (A.hi == 1.f && A.lo == 0.f) {
        each(BoolConst<true>{}, [&](float x, float y) {
            uint32_t xa, xb, ya, yb;
            cut(x, xa, xb);
            cut(fminf(x, fmaxf(y, 0.f)), ya, yb);
            a += xa - ya;
            b += xb - yb;
        }, [&](uint32_t) {
            sum += ((Fixed)(int)a << 22) + (int)b;
            a = b = 0;
        });
    } else {
        each(BoolConst<true>{}, [&](float x, float y) {
            float u, v;
            const bool some = exceeds(x, fminf(fmaxf(y, 0.f), 1.f), A, u, v);
            uint32_t xa, xb, ua, ub;
            cut(some ? x : 0.f, xa, xb);
            cut(some ? u : 0.f, ua, ub);
            a += xa - ua;
            b += xb - ub - (__float_as_uint((some ? v : 0.f) + kCut2) - kCut2Bits);
        }, [&](uint32_t) {
            sum += ((Fixed)(int)a << 22) + (int)b;
            a = b = 0;
        });
    }
    return warp_sum(sum);
}

// A barrier of the cluster in two parts, for all its threads: what lies between them overlaps the wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

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
__global__ void __launch_bounds__(kVerifyThreads, kVerifyBlocks) verify_drafts_kernel(const VerifyParams a) {
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
    cluster_arrive();  // this CTA runs: its shared memory may be written by the others (waited for in the first pass)
    const int n = (int)nn, V = a.vocab;
    const T *target = static_cast<const T *>(a.target) + (size_t)q0 * a.target_stride;
    const T *draft = a.draft ? static_cast<const T *>(a.draft) + (size_t)q0 * a.draft_stride : nullptr;
    const bool vec = a.vector_rows != 0;
    const float last_u = __ldg(a.final_uniforms + s);

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
                px = clean(prob(target + (size_t)up * a.target_stride, x));
                if (draft) qx = clean(prob(draft + (size_t)up * a.draft_stride, x));
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
    auto pass = [&](int node, Multiple A) -> Fixed {
        const Fixed mine = sum_residual<T, E>(target + (size_t)node * a.target_stride,
                                              draft ? draft + (size_t)node * a.draft_stride : nullptr, A, my_lo, my_hi,
                                              V, vec, lane);
        __syncthreads();  // (the last pass's sums have been read)
        if (lane == 0) sh.warp_sums[warp] = mine;
        __syncthreads();
        if (passes == 0) cluster_wait();
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
    Fixed taken = 0, Z = 0;   // A and the sum of r (known once `summed`), units of 2^-44
    Multiple A{0.f, 0.f};
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
        // u q Z < r; where r is p it is taken as it came
        const bool whole = draft ? taken == 0 : !gone(i);
        const Fixed have = draft && taken ? residual(sh.p[i], sh.q[i], A) : whole ? to_fixed(sh.p[i]) : 0;
        if (refusals ? below(sh.u[i], sh.q[i], Z, have) : below(sh.u[i], sh.q[i], whole ? sh.p[i] : 0.f)) {
            node = i;
            if (tid == 0) sh.path[count] = i;
            ++count;
            refusals = listed = 0;
            taken = Z = 0;
            A = {0.f, 0.f};
            summed = spent = false;
            continue;
        }
        if (spent) continue;  // (p and q are the same to the last bit: r stays what it was)
        if (draft) {
            const Fixed taken1 = refusals ? taken + Z : 1ll << 44;
            const Multiple A1 = to_multiple(taken1);
            const Fixed Z1 = pass(node, A1);
            if (Z1 <= 0) {
                spent = true;
                summed = false;   // (the warps' sums are those of nothing)
            } else {
                taken = taken1;
                A = A1;
                Z = Z1;
                summed = true;
                ++refusals;
            }
        } else {
            if (!summed) {
                Z = pass(node, A);
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
    if (Z <= 0) return;  // a row without a positive probability
    const T *prow = target + (size_t)node * a.target_stride;
    const T *qrow = draft ? draft + (size_t)node * a.draft_stride : nullptr;
    // floor(u Z), u in units of 2^-64
    const float u = fminf(fmaxf(last_u, 0.f), 0x1.fffffep-1f) * 0x1p32f;
    const uint32_t u_hi = __float2uint_rz(u), u_lo = __float2uint_rz((u - __uint2float_rz(u_hi)) * 0x1p32f);
    const Fixed goal = (Fixed)__umul64hi(((unsigned long long)u_hi << 32) | u_lo, (unsigned long long)Z);
    // without q: the refused tokens come off the sums of their stretches
    const int slot = (passes - 1) & 1;
    for (int j = tid; j < listed; j += kVerifyThreads) {
        const int i = sh.refused[j], w = sh.token[i] / per_warp;
        const unsigned long long off = 0ull - (unsigned long long)to_fixed(sh.p[i]);
        atomicAdd(reinterpret_cast<unsigned long long *>(&sh.cta_sum[slot][w / kVerifyWarps]), off);
        if (w / kVerifyWarps == rank) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.warp_sums[w % kVerifyWarps]), off);
    }
    __syncthreads();
    // Among `count` sums behind `below`: the one that goal falls into (-1: none), below moved up to it.
    auto find = [&](const Fixed *sums, int num, Fixed &below) -> int {
        const Fixed mine = lane < num ? sums[lane] : 0;
        Fixed upto = below + mine;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            const Fixed t = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += t - below;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, lane < num && goal < upto && goal >= upto - mine);
        if (hit == 0) return -1;
        below = __shfl_sync(0xffffffffu, upto - mine, __ffs(hit) - 1);
        return __ffs(hit) - 1;
    };
    static_assert(kVerifyWarps <= 16, "the scan above");
    Fixed below = 0;
    if (find(sh.cta_sum[slot], ctas, below) != rank) return;
    const int w = find(sh.warp_sums, kVerifyWarps, below);
    if (w < 0) return;
    const int w_lo = (rank * kVerifyWarps + w) * per_warp, w_hi = (int)min((long long)V, (long long)w_lo + per_warp);
    // the part of that warp's stretch, one to a warp
    const int f_lo = min(w_hi, w_lo + warp * per_fine), f_hi = min(w_hi, f_lo + per_fine);
    Fixed part = sum_residual<T, E>(prow, qrow, A, f_lo, f_hi, V, vec, lane);
    if (listed) {
        Fixed off = 0;
        for (int j = lane; j < listed; j += 32) {
            const int i = sh.refused[j];
            if (sh.token[i] >= f_lo && sh.token[i] < f_hi) off += to_fixed(sh.p[i]);
        }
        part -= warp_sum(off);
    }
    if (lane == 0) sh.fine[warp] = part;
    __syncthreads();
    if (find(sh.fine, kVerifyWarps, below) != warp) return;
    // its step and lane
    for (int v0 = f_lo; v0 < f_hi; v0 += kStep) {
        const int v = v0 + lane * E;
        float x[E], y[E];
        Fixed r[E], sum = 0;
        if (vec && v0 + kStep <= f_hi) {
            unpack_probs<T, E>(__ldg(reinterpret_cast<const uint4 *>(prow + v)), x);
            if (taken) unpack_probs<T, E>(__ldg(reinterpret_cast<const uint4 *>(qrow + v)), y);
        } else {
            load_probs<T, E>(prow, v, V, x);
            if (taken) load_probs<T, E>(qrow, v, V, y);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            r[e] = residual(x[e], taken ? y[e] : 0.f, A);
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
            // the first element whose running sum exceeds goal
            Fixed at = below + upto - sum;
            int pick = E;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (pick == E && goal >= at && goal < at + r[e]) pick = e;
                at += r[e];
            }
            const unsigned hit = __ballot_sync(0xffffffffu, pick < E);
            if (lane == __ffs(hit) - 1) a.next_tokens[s] = v + pick;
            return;
        }
        below += all;
    }
}

}  // namespace pkv
