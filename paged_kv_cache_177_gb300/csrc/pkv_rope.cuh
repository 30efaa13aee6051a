// pkv_rope.cuh -- the pass from the projections to the cache: the norm of
// every query and key head, their rotation to the token's position, and the
// write of queries, keys and values to where attention reads them.
#pragma once

#include "pkv_e4m3.cuh"
#include "pkv_prefill_tc.cuh"

namespace pkv {

struct RopeParams {
    void *q_out;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
    const void *q_weight, *k_weight;       // null: no norm
    const int64_t *positions;              // [num_axes][num_tokens]
    const float *inv_freq;                 // [rot / 2]
    const int32_t *axes;                   // [rot / 2] or null
    const int64_t *slots;
    void *k_cache, *v_cache;
    float eps;
    int num_axes, rot, num_tokens, num_q_heads, num_kv_heads, num_blocks;
    int warps_per_token;
};

// f / (2 pi), its whole turns off, as a 64-bit fraction of a turn, rounded down; |f| < 16 (every model's). With
// f = m 2^(e - 150), m its 24-bit significand, the product of m and 2^96 / (2 pi) only needs a shift.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
    constexpr unsigned __int128 kTurn = (unsigned __int128)0x28be60dbu << 64 | 0x9391054a7f09d5f4ull;  // 2^96 / (2 pi)
    const uint32_t bits = __float_as_uint(f) & 0x7fffffffu;
    const int e = max(1, (int)(bits >> 23));
    const uint32_t m = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);
    const int down = 182 - e;
    const uint64_t r = down >= 128 ? 0ull : (uint64_t)((kTurn * m) >> down);
    return f < 0.f ? 0ull - r : r;
}

// The same for any other finite f: f times 1 / (2 pi) as a sum of two doubles, the first product's rounding kept by a
// multiply-add, whole turns off each part; to the nearest, good to 2^-64 of a turn up to |f| = 2^40.
__device__ __noinline__ uint64_t turn_fraction_far(float f) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
    const double p = (double)f * kHi, hi = p - rint(p);
    double lo = fma((double)f, kHi, -p);
    lo = (lo - rint(lo)) + (double)f * kLo;
    lo -= rint(lo);
    return ((uint64_t)__double2ll_rn(hi * 0x1p63) << 1) + (uint64_t)__double2ll_rn(lo * 0x1p64);
}

// cos and sin of pos * f, NaN for a frequency that is not finite. The product is taken in turns and in integers, where
// whole turns fall off by themselves: the fraction is off by at most |pos| 2^-64 of a turn, and rounded to fp32
// once, so that a small angle has all its bits. (In fp64 it is as good, but this GPU's fp64 rate then bounds a
// decode step's few tokens: 6.4 us against 4.8 us for 64 of 48 heads.)
__device__ __forceinline__ float2 rotation(int64_t pos, float f) {
    const uint64_t per_position = fabsf(f) < 16.f ? turn_fraction(f) : turn_fraction_far(f);
    float turns = (float)(int64_t)((uint64_t)pos * per_position) * 0x1p-64f;
    if (!(fabsf(f) < INFINITY)) turns = __uint_as_float(0x7fc00000u);
    float2 cs;
    sincospif(2.f * turns, &cs.y, &cs.x);
    return cs;
}

// A lane's 8 consecutive elements of a row as loaded: 32-bit words.
template <typename T>
struct Raw8 {
    static constexpr int kWords = 2 * sizeof(T);
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
            reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __device__ __forceinline__ void pairs(uint64_t (&x)[4]) const {  // packed fp32 pairs, exact
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) x[i] = bf16x2_to_f2(w[i]);
            else x[i] = pack_f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 2) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
    }
};

// =====================================================================================
// A row is held by D / 8 neighbouring lanes, 8 elements each (16 bytes in bf16), so the mean square is
// a few shuffles and the other element of a half-split pair sits in the same place of the lane rot / 16
// further. A warp works on one token, 32 / (D / 8) rows at a time; a token's warps (one in a prompt, more
// in a decode step, where they are what keeps the SMs busy) share its rows.
//
// Norm and rotation are one multiply-add per element: with x' the pair's other element, w' its weight,
//   y = (x * w cos + x' * (-+) w' sin) / sqrt(mean x^2 + eps)
// and the two products of weight and angle belong to the lane's place in the row, not to the row: they
// are made once per token and kept in registers (the angles' fp32 sines and cosines once per warp, two
// a lane, through shared memory). So the pass is bound by its bytes: each row is read once and
// written once (16381 tokens of 48 heads of 128: bf16 71 us, 5.7 TB/s, fp32 129 us, 6.3 TB/s; keys and values into an e4m3
// cache 76 and 123 us, 4.8 and 5.7 TB/s).
// =====================================================================================
constexpr int kRopeWarps = 2;  // of a CTA (nothing is shared but the launch: eight took 75 us where two take 72)

template <typename T, int D, bool kInterleaved, bool kE4m3>
__global__ void __launch_bounds__(kRopeWarps * 32, 16) qk_norm_rope_append_kernel(const RopeParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes to a row, rows to a warp
    constexpr int kBatch = 8 / sizeof(T);       // row passes whose loads are in flight together: 64 bytes a lane
    constexpr int kTile = PKV_E4M3_TILE_BYTES(D);
    __shared__ float2 cs_s[kRopeWarps][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR, e0 = 8 * l;
    const int wpt = p.warps_per_token;
    const long long gw = (long long)blockIdx.x * kRopeWarps + warp;
    const int t = (int)(gw / wpt), wi = (int)(gw - (long long)t * wpt);
    if (t >= p.num_tokens) return;
    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads;
    int64_t slot = __ldg(p.slots + t);
    if (slot >= (int64_t)p.num_blocks * kBlock) {
        if (wi == 0 && lane == 0) raise_error(PKV_DEVERR_SLOT);
        slot = -1;
    }
    // Row pass i of a kind covers heads RPW i ..; the token's warps take the passes over the queries', then the
    // keys', then the values' heads in turn.
    const int q_passes = (Hq + RPW - 1) / RPW, kv_passes = slot < 0 ? 0 : (Hkv + RPW - 1) / RPW;
    Raw8<T> raw[kBatch];
    auto load = [&](const T *src, int i, int n, int heads) {  // passes i, i + wpt, ...
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int head = (i + b * wpt) * RPW + sub;
            if (i + b * wpt < n && head < heads) raw[b].load(src + (int64_t)head * D + e0);
        }
    };
    const T *q = static_cast<const T *>(p.q) + t * p.q_stride;
    load(q, wi, q_passes, Hq);  // on their way while the angles are made

    const int half = p.rot / 2;
    for (int i = lane; i < half; i += 32) {
        const int a = p.axes ? __ldg(p.axes + i) : 0;
        if (a < 0 || a >= p.num_axes) {
            if (t == 0 && wi == 0) raise_error(PKV_DEVERR_INDEX);
            cs_s[warp][i] = make_float2(1.f, 0.f);
        } else {
            cs_s[warp][i] = rotation(__ldg(p.positions + (int64_t)a * p.num_tokens + t), __ldg(p.inv_freq + i));
        }
    }
    __syncwarp();
    const bool turned = e0 < p.rot, first = e0 < half;
    const int shift = kInterleaved || !turned ? 0 : first ? half / 8 : -(half / 8);  // lanes to the pair's other element

    // the cache row of this token and a head
    auto cache_row = [&](void *cache, int head) {
        return static_cast<T *>(cache) + (((size_t)(slot >> 4) * Hkv + head) * kBlock + (slot & 15)) * D + e0;
    };
    auto quantised = [&](void *cache, int head, const float (&x)[8], bool live) {
        uint32_t sb;
        const uint2 codes = quantise8<LPR>(x, sb);
        if (live) {
            uint8_t *tile = static_cast<uint8_t *>(cache) + ((size_t)(slot >> 4) * Hkv + head) * kTile;
            *reinterpret_cast<uint2 *>(tile + (slot & 15) * D + e0) = codes;
            if (l == 0) tile[kBlock * D + (slot & 15)] = (uint8_t)sb;
        }
    };

    // the queries' or the keys' rows
    auto turn_rows = [&](auto keys_tag, const T *src, const T *weight, int i0, int n, int heads, bool loaded) {
        constexpr bool kKeys = decltype(keys_tag)::value;
        if (i0 >= n) return;
        // y = (x A + x' B) inv, in pairs of this lane's elements
        uint64_t A[4], B[4];
        {
            float w[8], wo[8];
            if (weight) {
                load8(weight + e0, w);
                load8(weight + e0 + 8 * shift, wo);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = wo[i] = 1.f;
            }
            float a[8], b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] = w[i];
                b[i] = 0.f;
                if (turned) {
                    const float2 c = cs_s[warp][kInterleaved ? (e0 + i) / 2 : (first ? e0 : e0 - half) + i];
                    const float other = kInterleaved ? w[i ^ 1] : wo[i];
                    const bool lead = kInterleaved ? (i & 1) == 0 : first;
                    a[i] = w[i] * c.x;
                    b[i] = (lead ? -other : other) * c.y;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                A[i] = pack_f2(a[2 * i], a[2 * i + 1]);
                B[i] = pack_f2(b[2 * i], b[2 * i + 1]);
            }
        }
        for (int i = i0; i < n; i += kBatch * wpt) {
            if (!loaded) load(src, i, n, heads);
            loaded = false;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (i + b * wpt >= n) break;
                const int head = (i + b * wpt) * RPW + sub;
                const bool live = head < heads;
                if (!live) {
#pragma unroll
                    for (int k = 0; k < Raw8<T>::kWords; ++k) raw[b].w[k] = 0u;
                }
                uint64_t x[4], o[4];
                raw[b].pairs(x);
                float inv = 1.f;
                if (weight) {
                    uint64_t s2 = 0;  // +0, +0
#pragma unroll
                    for (int k = 0; k < 4; ++k) s2 = fma_f2(x[k], x[k], s2);
                    float s0, s1;
                    unpack_f2(s2, s0, s1);
                    float ss = s0 + s1;
#pragma unroll
                    for (int w = LPR / 2; w > 0; w >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, w);
                    inv = rsqrtf(ss * (1.f / D) + p.eps);
                }
                if constexpr (kInterleaved) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float a0, a1;
                        unpack_f2(x[k], a0, a1);
                        o[k] = turned ? pack_f2(a1, a0) : 0ull;
                    }
                } else {
                    Raw8<T> r;
#pragma unroll
                    for (int k = 0; k < Raw8<T>::kWords; ++k) {
                        r.w[k] = __shfl_sync(0xffffffffu, raw[b].w[k], lane + shift);
                        if (!turned) r.w[k] = 0u;
                    }
                    r.pairs(o);
                }
                const uint64_t inv2 = pack_f2(inv, inv);
                float y[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t v = fma_f2(x[k], A[k], fma_f2(o[k], B[k], 0ull));
                    unpack_f2(fma_f2(v, inv2, 0ull), y[2 * k], y[2 * k + 1]);
                }
                if constexpr (kKeys && kE4m3) {
                    quantised(p.k_cache, head, y, live);
                } else if (live) {
                    store8(kKeys ? cache_row(p.k_cache, head)
                                 : static_cast<T *>(p.q_out) + ((size_t)t * Hq + head) * D + e0, y);
                }
            }
        }
    };
    turn_rows(BoolConst<false>{}, q, static_cast<const T *>(p.q_weight), wi, q_passes, Hq, true);
    int at = (wi + wpt - q_passes % wpt) % wpt;
    turn_rows(BoolConst<true>{}, static_cast<const T *>(p.k) + t * p.k_stride, static_cast<const T *>(p.k_weight), at,
              kv_passes, Hkv, false);
    at = (at + wpt - kv_passes % wpt) % wpt;
    const T *v = static_cast<const T *>(p.v) + t * p.v_stride;
    for (int i = at; i < kv_passes; i += kBatch * wpt) {
        load(v, i, kv_passes, Hkv);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (i + b * wpt >= kv_passes) break;
            const int head = (i + b * wpt) * RPW + sub;
            if constexpr (kE4m3) {
                float x[8];
                if (head >= Hkv) {
#pragma unroll
                    for (int k = 0; k < Raw8<T>::kWords; ++k) raw[b].w[k] = 0u;
                }
                raw[b].unpack(x);
                quantised(p.v_cache, head, x, head < Hkv);
            } else if (head < Hkv) {
                raw[b].store(cache_row(p.v_cache, head));
            }
        }
    }
}

}  // namespace pkv
