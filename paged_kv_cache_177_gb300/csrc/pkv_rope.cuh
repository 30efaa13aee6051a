// pkv_rope.cuh -- the pass from the projections to the cache: the norm of
// every query and key head, their rotation to the token's position, and the
// write of queries, keys and values to where attention reads them.
#pragma once

#include "pkv_e4m3.cuh"

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
};

// cos and sin of pos * f. The product is taken in turns and in 64 bits, where
// its whole turns come off without loss (an angle of 10^6 radians still has
// 2^-33 of a turn), then the rest goes through the fp32 functions.
__device__ __forceinline__ float2 rotation(int64_t pos, float f) {
    constexpr double kTurnsPerRadian = 0.15915494309189533577;
    double turns = (double)pos * (double)f * kTurnsPerRadian;
    turns -= rint(turns);
    float2 cs;
    sincospif(2.f * (float)turns, &cs.y, &cs.x);
    return cs;
}

// =====================================================================================
// One CTA per token: its rot / 2 rotations are computed once, into shared
// memory, and every head's row uses them. A row is held by D / 8 neighbouring
// lanes, 8 elements each (one 16-byte load in bf16), so the mean square is a
// few shuffles and a half-split pair's other element sits in the same place of
// the lane rot / 16 further. Bound by its bytes: each row is read once and
// written once.
// =====================================================================================
template <typename T, int D, bool kInterleaved, bool kE4m3>
__global__ void __launch_bounds__(256) qk_norm_rope_append_kernel(const RopeParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes to a row, rows to a warp
    constexpr int kTile = PKV_E4M3_TILE_BYTES(D);
    __shared__ float2 cs[D / 2];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int half = p.rot / 2;
    for (int i = tid; i < half; i += blockDim.x) {
        const int a = p.axes ? __ldg(p.axes + i) : 0;
        if (a < 0 || a >= p.num_axes) {
            if (t == 0) raise_error(PKV_DEVERR_INDEX);
            cs[i] = make_float2(1.f, 0.f);
        } else {
            cs[i] = rotation(__ldg(p.positions + (int64_t)a * p.num_tokens + t), __ldg(p.inv_freq + i));
        }
    }
    int64_t slot = __ldg(p.slots + t);
    if (slot >= (int64_t)p.num_blocks * kBlock) {
        if (tid == 0) raise_error(PKV_DEVERR_SLOT);
        slot = -1;
    }
    __syncthreads();
    const int l = tid % LPR, e0 = 8 * l;
    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    const int lane = tid & 31;
    // (rows are a warp's loop variable: every lane of a warp takes the same number of passes)
    for (int r0 = (tid >> 5) * RPW; r0 < rows; r0 += (blockDim.x >> 5) * RPW) {
        const int r = r0 + lane / LPR;
        const bool is_q = r < p.num_q_heads, is_k = !is_q && r < p.num_q_heads + p.num_kv_heads;
        const int h = is_q ? r : is_k ? r - p.num_q_heads : r - p.num_q_heads - p.num_kv_heads;
        const bool live = r < rows && (is_q || slot >= 0);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        if (live) {
            const T *src = static_cast<const T *>(is_q ? p.q : is_k ? p.k : p.v);
            load8(src + (int64_t)t * (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride) + h * D + e0, x);
        }
        const bool turned = is_q || is_k;
        if (p.q_weight) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (turned) {
                const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
                float w[8];
                load8(static_cast<const T *>(is_q ? p.q_weight : p.k_weight) + e0, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
            }
        }
        if constexpr (kInterleaved) {
            if (turned && e0 < p.rot) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 c = cs[e0 / 2 + i];
                    const float a = x[2 * i], b = x[2 * i + 1];
                    x[2 * i] = a * c.x - b * c.y;
                    x[2 * i + 1] = b * c.x + a * c.y;
                }
            }
        } else {
            const bool first = e0 < half;
            const int other = (lane & ~(LPR - 1)) | ((first ? l + p.rot / 16 : l - p.rot / 16) & (LPR - 1));
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], other);
            if (turned && e0 < p.rot) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 c = cs[(first ? e0 : e0 - half) + i];
                    x[i] = x[i] * c.x + (first ? -y[i] : y[i]) * c.y;
                }
            }
        }
        if (kE4m3) {
            uint32_t sb;
            const uint2 codes = quantise8<LPR>(x, sb);
            if (live && !is_q) {
                uint8_t *tile = static_cast<uint8_t *>(is_k ? p.k_cache : p.v_cache) +
                                ((size_t)(slot >> 4) * p.num_kv_heads + h) * kTile;
                *reinterpret_cast<uint2 *>(tile + (slot & 15) * D + e0) = codes;
                if (l == 0) tile[kBlock * D + (slot & 15)] = (uint8_t)sb;
            }
        }
        if (live && (is_q || !kE4m3)) {
            T *dst = is_q ? static_cast<T *>(p.q_out) + ((size_t)t * p.num_q_heads + h) * D
                          : static_cast<T *>(is_k ? p.k_cache : p.v_cache) +
                                (((size_t)(slot >> 4) * p.num_kv_heads + h) * kBlock + (slot & 15)) * D;
            store8(dst + e0, x);
        }
    }
}

}  // namespace pkv
