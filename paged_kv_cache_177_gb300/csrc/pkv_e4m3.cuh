// pkv_e4m3.cuh -- the cache in 8-bit floating point: quantising rows as they
// are written, reading blocks back, and decode attention over the tiles.
//
// A (block, kv head) tile is 16 rows of D e4m3 codes followed by the rows' 16
// scale bytes: element d of row r stands for code[r][d] * 2^(scale[r] - 127).
// The scale is a power of two (the least that brings the row's largest
// magnitude to at most 448, e4m3's largest value), so dividing by it is exact:
// a code is one rounding of the row's element and the same on every path that
// writes it. A floating-point code loses nothing to the coarser scale: its
// relative step is 2^-4 wherever in the range the element falls.
#pragma once

#include <cuda_fp16.h>

#include "pkv_kernels.cuh"

namespace pkv {

constexpr int kE4m3ExpLo = -50, kE4m3ExpHi = 50;  // range of a row's scale exponent

// Two floats to two e4m3 codes (a in the low byte), nearest even, saturating; NaN to NaN.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Two e4m3 codes (the low 16 bits) to two f16, exactly.
__device__ __forceinline__ uint32_t cvt_f16x2_e4m3x2(uint32_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
    return r;
}

// 2^(byte - 127): the scale a scale byte stands for (byte 0, never written by a quantiser, gives 0).
__device__ __forceinline__ float e8m0_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight consecutive elements of a row.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Quantises a row held 8 elements a lane by LPR neighbouring lanes (every lane of the warp
// calls it) and gives this lane's 8 codes and the row's scale byte. The exponent comes from the
// bits of the maximum: 448 = 1.75 * 2^8, so with max = f * 2^k, 1 <= f < 2, it is k - 8, one
// more where f > 1.75.
template <int LPR>
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], uint32_t &scale_byte) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[i]);
        top = fmaxf(top, a < INFINITY ? a : 0.f);  // NaN and infinities stay out
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t bits = __float_as_uint(top);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = bits == 0 ? 0 : max(kE4m3ExpLo, min(kE4m3ExpHi, e));
    scale_byte = (uint32_t)(e + 127);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fabsf(x[i]) < INFINITY ? x[i] * inv : __uint_as_float(0x7fc00000u);
    uint2 r;
    r.x = cvt_e4m3x2(y[0], y[1]) | (cvt_e4m3x2(y[2], y[3]) << 16);
    r.y = cvt_e4m3x2(y[4], y[5]) | (cvt_e4m3x2(y[6], y[7]) << 16);
    return r;
}

// =====================================================================================
// Append: D / 8 lanes to a (token, kv head) row of K and the same row of V, 8 elements a lane.
// Bound by its bytes (and by the launch for a decode step's few rows).
// =====================================================================================
template <typename T, int D>
__global__ void __launch_bounds__(256)
    kv_append_e4m3_kernel(const T *__restrict__ k, const T *__restrict__ v, const int64_t *__restrict__ slots,
                          uint8_t *__restrict__ kc, uint8_t *__restrict__ vc, int num_tokens, int num_kv_heads,
                          int num_blocks) {
    constexpr int LPR = D / 8;
    constexpr int kTile = PKV_E4M3_TILE_BYTES(D);
    const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / LPR;
    const int l = threadIdx.x % LPR;
    bool live = row < (long long)num_tokens * num_kv_heads;
    const int t = live ? (int)(row / num_kv_heads) : 0;
    const int h = (int)(row - (long long)t * num_kv_heads);
    int64_t slot = live ? __ldg(slots + t) : -1;
    if (slot >= (int64_t)num_blocks * kBlock) {
        if (h == 0 && l == 0) raise_error(PKV_DEVERR_SLOT);
        slot = -1;
    }
    live = slot >= 0;
    float x[2][8];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = 0.f;
        if (live) load8((c ? v : k) + row * D + 8 * l, x[c]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t sb;
        const uint2 codes = quantise8<LPR>(x[c], sb);
        if (live) {
            uint8_t *tile = (c ? vc : kc) + ((size_t)(slot >> 4) * num_kv_heads + h) * kTile;
            *reinterpret_cast<uint2 *>(tile + (slot & 15) * D + 8 * l) = codes;
            if (l == 0) tile[kBlock * D + (slot & 15)] = (uint8_t)sb;
        }
    }
}

// =====================================================================================
// Reading back: one CTA per (pair, kv head); 2 D threads take 8 codes each of the K tile's
// 16 D, then of the V tile's.
// =====================================================================================
template <typename T, int D>
__global__ void __launch_bounds__(2 * D)
    dequantize_blocks_kernel(T *__restrict__ dk, T *__restrict__ dv, const uint8_t *__restrict__ sk,
                             const uint8_t *__restrict__ sv, const int64_t *__restrict__ pairs, int num_kv_heads,
                             int src_num_blocks, int dst_num_blocks) {
    constexpr int kTile = PKV_E4M3_TILE_BYTES(D);
    const int64_t src = __ldg(pairs + 2 * (int64_t)blockIdx.x), dst = __ldg(pairs + 2 * (int64_t)blockIdx.x + 1);
    const int h = blockIdx.y, tid = threadIdx.x;
    if (src < 0 || src >= src_num_blocks || dst < 0 || dst >= dst_num_blocks) {
        if (h == 0 && tid == 0) raise_error(PKV_DEVERR_PAIR);
        return;
    }
    const size_t from = ((size_t)src * num_kv_heads + h) * kTile, to = ((size_t)dst * num_kv_heads + h) * kBlock * D;
    uint2 c[2];
    uint32_t sb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint8_t *tile = (i ? sv : sk) + from;
        c[i] = *reinterpret_cast<const uint2 *>(tile + 8 * tid);
        sb[i] = tile[kBlock * D + 8 * tid / D];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float scale = e8m0_value(sb[i]);
        float x[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t w = cvt_f16x2_e4m3x2((q < 2 ? c[i].x : c[i].y) >> (16 * (q & 1)));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
            x[2 * q] = f.x * scale;
            x[2 * q + 1] = f.y * scale;
        }
        store8((i ? dv : dk) + to + 8 * tid, x);
    }
}

// =====================================================================================
// Decode, one warp per (sequence, query head): 32 tokens at a time, a lane scores one of them;
// then every lane sums D / 32 elements of the output over the 32 weights.
// =====================================================================================
template <int D, typename OutT>
__global__ void __launch_bounds__(128) decode_e4m3_kernel(const DecodeParams p) {
    constexpr int kTile = PKV_E4M3_TILE_BYTES(D), PER = D / 32;
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hq = blockIdx.x * 4 + warp, s = blockIdx.y;
    if (hq >= p.num_q_heads) return;
    const int h = hq / p.group;
    const int len = seq_len(p, s, lane == 0 && hq == 0);
    const size_t row = (size_t)s * p.num_q_heads + hq;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + row * D;
    for (int i = lane; i < D; i += 32) qs[warp][i] = __bfloat162float(q[i]) * p.scale_log2;
    __syncwarp();
    const uint8_t *kc = static_cast<const uint8_t *>(p.k_cache), *vc = static_cast<const uint8_t *>(p.v_cache);
    const int32_t *table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    auto code_value = [](uint8_t c) {
        const uint32_t w = cvt_f16x2_e4m3x2(c);
        return __half2float(__ushort_as_half((unsigned short)w));
    };
    for (int t0 = 0; t0 < len; t0 += 32) {
        const int t = t0 + lane;
        int pb = -1;
        if (t < len) {
            pb = __ldg(table + t / kBlock);
            if (pb < 0 || pb >= p.num_blocks) {
                raise_error(PKV_DEVERR_BLOCK_ID);
                pb = -1;
            }
        }
        float x = t < len ? 0.f : -INFINITY;  // a bad block reads as zeros
        if (pb >= 0) {
            const uint8_t *tile = kc + ((size_t)pb * p.num_kv_heads + h) * kTile;
            float dot = 0.f;
            for (int d = 0; d < D; ++d) dot = fmaf(code_value(tile[(t & 15) * D + d]), qs[warp][d], dot);
            x = dot * e8m0_value(tile[kBlock * D + (t & 15)]);
        }
        float mx = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m, mx), al = exp2f(m - mn), w = exp2f(x - mn);
        m = mn;
        l = l * al + w;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] *= al;
        for (int i = 0; i < min(32, len - t0); ++i) {
            const int b = __shfl_sync(0xffffffffu, pb, i);
            const float wi = __shfl_sync(0xffffffffu, w, i);
            if (b < 0) continue;
            const uint8_t *tile = vc + ((size_t)b * p.num_kv_heads + h) * kTile;
            const int r = (t0 + i) & 15;
            const float ws = wi * e8m0_value(tile[kBlock * D + r]);
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(code_value(tile[r * D + lane + 32 * e]), ws, acc[e]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    OutT *out = static_cast<OutT *>(p.out) + row * D;
    const float inv = len > 0 ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) out[lane + 32 * e] = to_out<OutT>(acc[e] * inv);
}

}  // namespace pkv
