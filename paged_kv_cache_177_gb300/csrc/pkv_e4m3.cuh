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

#include "pkv_cursor.cuh"
#include "pkv_kernels.cuh"

namespace pkv {

template <int N>
struct IntConst {  // a compile-time number passed to a generic lambda
    static constexpr int value = N;
};

constexpr int kE4m3ExpLo = -50, kE4m3ExpHi = 50;  // range of a row's scale exponent

// The decode kernel's reference for the weights' exponents: set kE4m3RefSet under the largest, moved when one passes
// kE4m3RefUp. kE4m3LeastByte stands for 2^-64, what a value row without magnitude takes there: lower than any
// quantiser's, so that the row does not lift the reference, and high enough that its weight, which fp32 holds
// down to 2^-126, adds to the sum all that counts beside the 2^-39 that a row of the largest scale adds at least.
// (With a row of zeros far above all other scores the others' weights do lose bits, from where their share of the weight
// is below 2^-(89 + ev), ev the exponent of their values: outputs that much smaller than the values.)
constexpr float kE4m3RefSet = 11.f, kE4m3RefUp = 15.5f;
constexpr uint32_t kE4m3LeastByte = 127 - 64;

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
// more where f > 1.75. NaN stays out of a maximum and becomes a NaN code by itself; rows that hold
// infinities are told by their maximum and go around again with NaN in their place (with a look at
// every element, the append of 16393 tokens of 40 heads was bound by the ALU: 101 us, 81 us so).
template <int LPR>
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], uint32_t &scale_byte) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    auto row_max = [&]() {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) top = max3f(top, fabsf(y[i]), fabsf(y[i + 1]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        return top;
    };
    float top = row_max();
    if (__builtin_expect(__any_sync(0xffffffffu, top == INFINITY), 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fabsf(y[i]) < INFINITY ? y[i] : __uint_as_float(0x7fc00000u);
        top = row_max();
    }
    const uint32_t bits = __float_as_uint(top);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = bits == 0 ? 0 : max(kE4m3ExpLo, min(kE4m3ExpHi, e));
    scale_byte = (uint32_t)(e + 127);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint2 r;
    r.x = cvt_e4m3x2(y[0] * inv, y[1] * inv) | (cvt_e4m3x2(y[2] * inv, y[3] * inv) << 16);
    r.y = cvt_e4m3x2(y[4] * inv, y[5] * inv) | (cvt_e4m3x2(y[6] * inv, y[7] * inv) << 16);
    return r;
}

// =====================================================================================
// Append: D / 8 lanes to a (token, kv head) row of K and the same row of V, 8 elements a lane; a CTA takes the
// rows of one head and 16 (D = 128) or 32 tokens: tokens mostly come in slot order, and then their rows and
// scale bytes fill whole tiles (by token with all heads, a tile's pieces came from 16 CTAs and took 17% more).
// Bound by its bytes (16393 tokens of 40 heads, bf16: 81 us, 6.2 TB/s), and by the launch for a decode step's few rows.
// =====================================================================================
constexpr int kAppendThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads)
    kv_append_e4m3_kernel(const T *__restrict__ k, const T *__restrict__ v, const int64_t *__restrict__ slots,
                          uint8_t *__restrict__ kc, uint8_t *__restrict__ vc, int num_tokens, int num_kv_heads,
                          int num_blocks) {
    constexpr int LPR = D / 8;
    constexpr int kTile = PKV_E4M3_TILE_BYTES(D);
    const int l = threadIdx.x % LPR, h = blockIdx.y;
    const long long t = (long long)blockIdx.x * (kAppendThreads / LPR) + threadIdx.x / LPR;
    int64_t slot = t < num_tokens ? __ldg(slots + t) : -1;
    float x[2][8];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = 0.f;
        if (t < num_tokens) load8((c ? v : k) + (t * num_kv_heads + h) * D + 8 * l, x[c]);
    }
    if (slot >= (int64_t)num_blocks * kBlock) {
        if (h == 0 && l == 0) raise_error(PKV_DEVERR_SLOT);
        slot = -1;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t sb;
        const uint2 codes = quantise8<LPR>(x[c], sb);
        if (slot >= 0) {
            uint8_t *tile = (c ? vc : kc) + ((size_t)(slot >> 4) * num_kv_heads + h) * kTile;
            *reinterpret_cast<uint2 *>(tile + (slot & 15) * D + 8 * l) = codes;
            if (l == 0) tile[kBlock * D + (slot & 15)] = (uint8_t)sb;
        }
    }
}

// =====================================================================================
// Reading back: grid (parts of a block, pairs, K / V). A block's tiles of all heads are one run in both caches; a
// thread takes 16 codes of it (more a thread, or both caches, measured slower by 7 of 184 us for a prompt's append
// and read-back, 13 x 1261 tokens of 40 heads).
// =====================================================================================
constexpr int kReadBackThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kReadBackThreads)
    dequantize_blocks_kernel(T *__restrict__ dk, T *__restrict__ dv, const uint8_t *__restrict__ sk,
                             const uint8_t *__restrict__ sv, const int64_t *__restrict__ pairs, int num_pairs,
                             int num_kv_heads, int src_num_blocks, int dst_num_blocks) {
    constexpr int kTile = PKV_E4M3_TILE_BYTES(D);
    const int i = blockIdx.x * kReadBackThreads + threadIdx.x;  // 16-code piece of the block: D to a tile
    const int h = i / D, u = i % D;
    const bool live = h < num_kv_heads;
    for (int pr = blockIdx.y; pr < num_pairs; pr += gridDim.y) {
        const int64_t src = __ldg(pairs + 2 * (int64_t)pr), dst = __ldg(pairs + 2 * (int64_t)pr + 1);
        if (src < 0 || src >= src_num_blocks || dst < 0 || dst >= dst_num_blocks) {
            if (i == 0 && blockIdx.z == 0) raise_error(PKV_DEVERR_PAIR);
            continue;
        }
        if (!live) continue;
        const size_t from = ((size_t)src * num_kv_heads + h) * kTile;
        const size_t to = (size_t)dst * num_kv_heads * kBlock * D + (size_t)16 * i;
        const uint8_t *tile = (blockIdx.z ? sv : sk) + from;
        const uint4 c = *reinterpret_cast<const uint4 *>(tile + 16 * u);
        const float scale = e8m0_value(tile[kBlock * D + 16 * u / D]);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float x[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t f2 = cvt_f16x2_e4m3x2(w[2 * half + (q >> 1)] >> (16 * (q & 1)));
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&f2));
                x[2 * q] = f.x * scale;
                x[2 * q + 1] = f.y * scale;
            }
            store8((blockIdx.z ? dv : dk) + to + 8 * half, x);
        }
    }
}

// =====================================================================================
// Decode over e4m3 tiles. The decomposition is the persistent bf16 kernel's: one CTA per SM,
// NW warps, each an independent worker with its own ring of NS stages; all (sequence, kv head)
// units' blocks form one line of T positions, cut into equal ranges, one per worker.
//
// The step over staged (K, V) blocks, for the group's query heads as the MMA's N:
//   x_t = (scale log2 e) 2^(ek_t + eq) <codes K_t, q'>      q = q' 2^eq, q' in f16
//   y_t = x_t + ev_t;   w_t = 2^(y_t - m)
//   l = sum_t w_t 2^-ev_t;   O = sum_t w_t codes V_t
// and the output is O / l. Codes widen to f16 without loss, and products with a query of 8
// significant bits are exact in the tensor cores' fp32 sums, so no code is multiplied by its scale:
// K's enters the score, V's the exponent of the weight. The reference m follows y, not x, so the
// weights -- the one thing rounded here, to f16's 11 bits -- are largest where their values
// matter most, whatever the rows' scales. m lies 2^11 to 2^15.5 (kE4m3RefUp, below f16's largest value)
// under the largest y so far: a weight has its 11 bits down to 2^-25 of the largest, and what is lost
// below f16's last step is at most 2^-36 of the largest w |codes| a row. O and l take the same w, each
// before or after its rounding, so a score so large that fp32 cannot add ev to it moves both alike.
// A row's exponent lies in [-50, 50], so l neither overflows nor loses a term that counts.
//
// That holds as long as a row's scale says how large its values are. It does not for a row of zeros, whose
// scale byte is 127 as if it held values up to 448: it would lift m over the rows that make up O. Blocks
// with a byte 127 in them are looked at (a warp's vote), and rows without magnitude (zeros, or NaN and
// zeros) take kE4m3LeastByte. So do bytes below it, which no quantiser writes: 0, the scale of every row
// that nothing was written to, is one. (Values of size 224 to 448 have the byte too: a cache of nothing else takes 148 us
// where 119 do, 256 contexts around 1000 of 8 heads.)
//
// A tile, codes and scales, is one contiguous run of 16 (D + 1) bytes and comes by one untiled bulk
// copy: the runs start at any multiple of 16 bytes, and a tiled copy of 128-byte rows from such a
// start asks L2 for two lines a row (with the arithmetic left out it took 124 us where the
// bulk copies took 115 us on 256 sequences of 8 heads, 715 MB). So the rows lie in shared memory
// as in the cache, and fragments are read 16 bytes a lane in the order the MMAs can take them:
//   K: lane t4 holds chunks t4 and t4 + 4 of its token's row, four codes of each for every MMA (the order of
//      a contraction is free as long as q's fragment has it too);
//   V: lane (gq, t4) holds codes (D/8) gq .. of tokens 2 t4, + 1, + 8, + 9; a byte permutation pairs
//      two tokens' codes of one element, and the MMAs' rows take the lane's elements two by two.
// These reads meet two- and four-way bank conflicts, 96 shared-memory cycles a block (D = 128) of the
// about 170 that its bytes take from HBM at one SM's share.
// =====================================================================================
template <int D, int NT>
struct WarpAttnE4m3 {
    static constexpr int kMmas = D / 16;     // of a block's QK^T, and of its PV
    static constexpr int kOwn = D / 8;       // output elements of a lane, per head
    static constexpr int kParts = D / 64;    // 16-byte chunks of a K row that a lane holds
    using QRaw = uint4[kParts][2][NT];       // q[head gq][64 j + 16 t4 .. + 15], bf16
    float m[NT][2], l[NT][2], qs[NT][2];     // of heads 2 t4, 2 t4 + 1 of each 8 columns; qs: score scale, log2 domain
    float acc[kMmas][NT][4];                 // [i][.][e]: head 2 t4 + (e & 1), element kOwn gq + 2 i + (e >> 1)
    uint32_t qf[kMmas][NT][2];

    static __device__ __forceinline__ void load_raw(QRaw &raw, const __nv_bfloat16 *q_group, int g, int lane) {
        const int gq = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int hl = nt * 8 + gq;
            const uint4 *row = reinterpret_cast<const uint4 *>(q_group + (size_t)(hl < g ? hl : 0) * D + 16 * t4);
#pragma unroll
            for (int j = 0; j < kParts; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    raw[j][i][nt] = hl < g ? __ldg(row + 8 * j + i) : make_uint4(0u, 0u, 0u, 0u);
        }
    }

    // q to f16, each head scaled by a power of two that brings its largest element to [2^13, 2^14):
    // exact down to 2^-27 of that element.
    __device__ __forceinline__ void set_q(const QRaw &raw, float scale_log2, int lane) {
        const int t4 = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float top = 0.f;
            auto each = [&](auto f) {
#pragma unroll
                for (int j = 0; j < kParts; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w[4] = {raw[j][i][nt].x, raw[j][i][nt].y, raw[j][i][nt].z, raw[j][i][nt].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // elements 64 j + 16 t4 + 8 i + 2 k, + 1
                            f(4 * j + 2 * i + (k >> 1), k & 1, __uint_as_float(w[k] << 16),
                              __uint_as_float(w[k] & 0xffff0000u));
                    }
            };
            each([&](int, int, float a, float b) {
                a = fabsf(a), b = fabsf(b);
                top = fmaxf(top, fmaxf(a < INFINITY ? a : 0.f, b < INFINITY ? b : 0.f));
            });
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // exponent of the scale, kept where both it and its reciprocal are normal numbers
            const int e = top > 0.f ? max(-100, min(113, (int)(__float_as_uint(top) >> 23) - 127 - 13)) : 0;
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
            each([&](int mma, int r, float a, float b) {
                const __half2 h = __floats2half2_rn(a * inv, b * inv);
                qf[mma][nt][r] = *reinterpret_cast<const uint32_t *>(&h);
            });
            const float sc = __uint_as_float((uint32_t)(127 + e) << 23) * scale_log2;  // of head gq
            qs[nt][0] = __shfl_sync(0xffffffffu, sc, 8 * t4);
            qs[nt][1] = __shfl_sync(0xffffffffu, sc, 8 * t4 + 4);
        }
    }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < kMmas; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
        }
    }

    // Bits 2 r and 2 r + 1: whether row r of the tile at this shared address has a code that is neither zero nor NaN in its
    // first and second half.
    static __device__ __noinline__ uint32_t rows_with_magnitude(uint32_t tile, int lane) {
        uint32_t some = 0;
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
            uint32_t c[4];
            ld_shared_v4(tile + lane * (D / 2) + 16 * i, c);
#pragma unroll
            for (int w = 0; w < 4; ++w) some |= ((c[w] & 0x7f7f7f7fu) + 0x01010101u) & 0x7e7e7e7eu;
        }
        return __ballot_sync(0xffffffffu, some != 0);
    }

    // NB staged blocks of one unit: one softmax update, and enough independent MMAs to keep the
    // tensor pipe fed from three or four warps a scheduler. Rows of the last block from `valid` on are not
    // tokens. tile: shared address of each block's K tile, its V tile one tile further.
    template <int NB>
    __device__ __forceinline__ void blocks(const uint32_t (&tile)[NB], int valid, int lane) {
        constexpr int kTile = PKV_E4M3_TILE_BYTES(D);
        const int gq = lane >> 2, t4 = lane & 3;
        float sc[NB][NT][4], sb[NB][NT][4];
        uint32_t kb[NB][2], vb[NB][2];  // scale bytes of this lane's two token rows gq and gq + 8
        bool look = false;              // a value row may be without magnitude
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t at = tile[b] + kBlock * D + gq;
            kb[b][0] = ld_shared_u8(at), kb[b][1] = ld_shared_u8(at + 8);
            vb[b][0] = ld_shared_u8(at + kTile), vb[b][1] = ld_shared_u8(at + kTile + 8);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                look |= vb[b][i] == 127u;
                // (253: the largest exponent whose 2^-ev is a normal number; past the end a row's byte may be any)
                vb[b][i] = max(kE4m3LeastByte, min(253u, vb[b][i]));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[b][nt][e] = sb[b][nt][e] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kParts; ++j)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t k0[4], k1[4];
                const uint32_t at = tile[b] + gq * D + 64 * j + 16 * t4;
                ld_shared_v4(at, k0);
                ld_shared_v4(at + 8 * D, k1);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t a[4] = {cvt_f16x2_e4m3x2(k0[w]), cvt_f16x2_e4m3x2(k1[w]),
                                           cvt_f16x2_e4m3x2(k0[w] >> 16), cvt_f16x2_e4m3x2(k1[w] >> 16)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16_16816(w & 1 ? sb[b][nt] : sc[b][nt], a, qf[4 * j + w][nt][0], qf[4 * j + w][nt][1]);
                }
            }
        if (__builtin_expect(__any_sync(0xffffffffu, look), 0)) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t rows = rows_with_magnitude(tile[b] + kTile, lane);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (!(rows >> (2 * (gq + 8 * i)) & 3u)) vb[b][i] = kE4m3LeastByte;
            }
        }
        float kv[NB][2], ev[NB][2], un[NB][2];  // 2^ek, ev, 2^-ev
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                kv[b][i] = e8m0_value(kb[b][i]);
                ev[b][i] = __uint_as_float(0x4b000000u | vb[b][i]) - (8388608.f + 127.f);  // byte - 127
                un[b][i] = e8m0_value(254u - vb[b][i]);
            }
        uint32_t p0[NB][NT], p1[NB][NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float y[NB][4], mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[b][e] = fmaf((sc[b][nt][e] + sb[b][nt][e]) * kv[b][e >> 1], qs[nt][e & 1], ev[b][e >> 1]);
                    if (b == NB - 1 && gq + 8 * (e >> 1) >= valid) y[b][e] = -INFINITY;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) mx[c] = max3f(mx[c], y[b][c], y[b][c + 2]);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                for (int c = 0; c < 2; ++c) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], o));
            if (__any_sync(0xffffffffu, mx[0] - m[nt][0] > kE4m3RefUp || mx[1] - m[nt][1] > kE4m3RefUp)) {  // (seldom)
                float al[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float to = m[nt][c];
                    if (mx[c] - to > kE4m3RefUp) {
                        to = mx[c] - kE4m3RefSet;
                        if (mx[c] - to > kE4m3RefUp) to = mx[c];  // the step of fp32 is larger than that
                    }
                    al[c] = to == m[nt][c] ? 1.f : ex2_approx(m[nt][c] - to);
                    m[nt][c] = to;
                    l[nt][c] *= al[c];
                }
#pragma unroll
                for (int i = 0; i < kMmas; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][nt][e] *= al[e & 1];
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = ex2_approx(y[b][e] - m[nt][e & 1]);
                    l[nt][e & 1] = fmaf(w[e], un[b][e >> 1], l[nt][e & 1]);
                }
                const __half2 w0 = __floats2half2_rn(w[0], w[1]), w1 = __floats2half2_rn(w[2], w[3]);
                p0[b][nt] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&w0));
                p1[b][nt] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&w1));
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            constexpr int kWords = kOwn / 4;
            uint32_t v[4][kWords];  // tokens 2 t4, + 1, + 8, + 9
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t at = tile[b] + kTile + (2 * t4 + (r & 1) + 8 * (r >> 1)) * D + kOwn * gq;
                if constexpr (kWords == 4) ld_shared_v4(at, v[r]);
                else ld_shared_v2(at, v[r]);
            }
            if (b == NB - 1 && valid < kBlock) {  // what is not a token may hold anything: no weight undoes a NaN
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (2 * t4 + (r & 1) + 8 * (r >> 1) >= valid) {
#pragma unroll
                        for (int w = 0; w < kWords; ++w) v[r][w] = 0u;
                    }
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t lo = __byte_perm(v[0][w], v[1][w], e ? 0x7362 : 0x5140);
                    const uint32_t hi = __byte_perm(v[2][w], v[3][w], e ? 0x7362 : 0x5140);
                    const uint32_t a[4] = {cvt_f16x2_e4m3x2(lo), cvt_f16x2_e4m3x2(lo >> 16), cvt_f16x2_e4m3x2(hi),
                                           cvt_f16x2_e4m3x2(hi >> 16)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[2 * w + e][nt], a, p0[b][nt], p1[b][nt]);
                }
        }
    }

    // Sums l over the 8 lanes that share each head column.
    __device__ __forceinline__ void reduce_l() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], o);
    }

    // The g heads' outputs (after reduce_l) into rows [g][D], or their (max, sum, acc) states into [g][2 + D].
    template <typename OutT>
    __device__ __forceinline__ void store_rows(OutT *rows, int g, int lane) const {
        const int gq = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int head = nt * 8 + 2 * t4 + e;
                if (head >= g) continue;
                const float inv = 1.f / l[nt][e];
#pragma unroll
                for (int i = 0; i < kMmas; i += 4) {
                    float o[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        o[2 * k] = acc[i + k][nt][e] * inv;
                        o[2 * k + 1] = acc[i + k][nt][e + 2] * inv;
                    }
                    store8(rows + (size_t)head * D + kOwn * gq + 2 * i, o);
                }
            }
    }
    __device__ __forceinline__ void store_state(float *slot, int g, int lane) const {
        const int gq = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int head = nt * 8 + 2 * t4 + e;
                if (head >= g) continue;
                float *row = slot + (size_t)head * (2 + D);
                if (gq == 0) {
                    row[0] = m[nt][e];
                    row[1] = l[nt][e];
                }
#pragma unroll
                for (int i = 0; i < kMmas; ++i)
                    *reinterpret_cast<float2 *>(row + 2 + kOwn * gq + 2 * i) =
                        make_float2(acc[i][nt][e], acc[i][nt][e + 2]);
            }
    }
};

template <int D, int NS, int NW>
struct E4m3Cfg {
    static constexpr int kTile = PKV_E4M3_TILE_BYTES(D);
    static constexpr int kStage = 2 * kTile;  // K, then V
    static constexpr int kThreads = NW * 32;
    static constexpr int kBarOff = NW * NS * kStage;
    static constexpr int kPrefixOff = kBarOff + NW * NS * 8;
    static constexpr size_t smem_bytes(int num_seqs) { return kPrefixOff + (size_t)(num_seqs + 1) * 4; }
    static_assert((NS & (NS - 1)) == 0, "stage index");
    static_assert(kStage % 16 == 0, "bulk copies start on 16 bytes");
};

// A unit cut by the end of the range of the worker that began it: its segments (0: not cut), that worker,
// and its first output row. One record a unit where units are fewer than workers, else one a worker.
struct E4m3Cut {
    int segments, worker, row, pad;
};

template <int D, int NT, int NB, int NS, int NW, typename OutT>
__global__ void __launch_bounds__(NW * 32, 1)
    decode_e4m3_kernel(const DecodeParams p, E4m3Cut *cuts, const int whole_units, const int cuts_by_unit) {
    using C = E4m3Cfg<D, NS, NW>;
    using WA = WarpAttnE4m3<D, NT>;
    extern __shared__ __align__(16) uint8_t base[];
    __shared__ int warp_total[NW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.num_seqs, Hkv = p.num_kv_heads, g = p.group;
    uint64_t *full = reinterpret_cast<uint64_t *>(base + C::kBarOff) + warp * NS;
    int *prefix = reinterpret_cast<int *>(base + C::kPrefixOff);
    OutT *out = static_cast<OutT *>(p.out);
    if (tid == 0) {
        for (int i = 0; i < NW * NS; ++i) mbar_init(full + i, 1);
        mbar_fence_init();
    }

    // block counts of the sequences, summed up to each (every CTA makes its own copy)
    const int per = (S + C::kThreads - 1) / C::kThreads;
    const int s_lo = min(S, tid * per), s_hi = min(S, s_lo + per);
    int local = 0;
    for (int s = s_lo; s < s_hi; ++s) local += (seq_len(p, s, blockIdx.x == 0) + kBlock - 1) / kBlock;
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    int run = incl - local;
    for (int w = 0; w < warp; ++w) run += warp_total[w];
    for (int s = s_lo; s < s_hi; ++s) {
        prefix[s] = run;
        run += (seq_len(p, s, false) + kBlock - 1) / kBlock;
    }
    if (tid == 0) {
        int tot = 0;
        for (int w = 0; w < NW; ++w) tot += warp_total[w];
        prefix[S] = tot;
    }
    __syncthreads();
    pdl_trigger();  // the merge may be set up; it waits for the states

    for (int s = blockIdx.x; s < S; s += gridDim.x)  // empty contexts: zero rows
        if (prefix[s + 1] == prefix[s]) {
            OutT *o = out + (size_t)s * p.num_q_heads * D;
            for (int i = tid; i < p.num_q_heads * D; i += C::kThreads) o[i] = to_out<OutT>(0.f);
            if (cuts_by_unit)
                for (int h = tid; h < Hkv; h += C::kThreads) cuts[s * Hkv + h].segments = 0;
        }

    // this worker's range of positions: an equal share, of no less than its ring holds, or (short contexts) a share of whole units
    const long long T = (long long)Hkv * prefix[S];
    const int all = gridDim.x * NW, w = blockIdx.x * NW + warp;
    const long long U = (long long)S * Hkv;
    const int W = (int)min((long long)all, whole_units ? U : max(1LL, T / NS));
    long long start = 0, end = 0;
    if (w < W) {
        auto unit_begin = [&](long long u) {
            const int s = (int)(u / Hkv), h = (int)(u - (long long)s * Hkv);
            return u >= U ? T : (long long)Hkv * prefix[s] + (long long)h * (prefix[s + 1] - prefix[s]);
        };
        start = whole_units ? unit_begin(U * w / W) : T * w / W;
        end = whole_units ? unit_begin(U * (w + 1) / W) : T * (w + 1) / W;
    }
    const int cnt = (int)(end - start);
    if (cnt <= 0) {
        if (cuts && !cuts_by_unit && lane == 0) cuts[w].segments = 0;
        return;
    }
    Cursor c;
    {
        int lo = 0, hi = S - 1;  // largest s with Hkv * prefix[s] <= start (never an empty sequence)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((long long)Hkv * prefix[mid] <= start) lo = mid; else hi = mid - 1;
        }
        c.s = lo;
        c.n = prefix[lo + 1] - prefix[lo];
        const int r = (int)(start - (long long)Hkv * prefix[lo]);
        c.h = r / c.n;
        c.j = r - c.h * c.n;
    }

    // Block ids of 32 positions (lane i: the i-th from the cursor), gathered a batch ahead of use,
    // each with its kv head.
    struct Batch {
        int pb, h;
    };
    auto batch_of = [&](Cursor b, int count) -> Batch {
        Batch r{0, 0};
        if (lane < count) {
            cursor_advance(b, lane, prefix, Hkv);
            r.pb = __ldg(p.block_tables + (size_t)b.s * p.max_blocks_per_seq + b.j);
            r.h = b.h;
        }
        return r;
    };
    Cursor bnext = c;
    Batch cur = batch_of(c, min(32, cnt)), nxt{0, 0};
    if (cnt > 32) {
        cursor_advance(bnext, 32, prefix, Hkv);
        nxt = batch_of(bnext, min(32, cnt - 32));
    }
    uint8_t *ring = base + warp * NS * C::kStage;
    const uint64_t policy = l2_evict_first();
    int issued = 0;
    auto issue = [&]() {
        if (issued > 0 && (issued & 31) == 0) {
            cur = nxt;
            if (issued + 32 < cnt) {
                cursor_advance(bnext, 32, prefix, Hkv);
                nxt = batch_of(bnext, min(32, cnt - issued - 32));
            }
        }
        const int pb = __shfl_sync(0xffffffffu, cur.pb, issued & 31);
        const int h = __shfl_sync(0xffffffffu, cur.h, issued & 31);
        const int st = issued & (NS - 1);
        uint8_t *stage = ring + st * C::kStage;
        if (pb >= 0 && pb < p.num_blocks) {
            if (lane == 0) {
                const size_t from = ((size_t)pb * Hkv + h) * C::kTile;
                mbar_arrive_expect_tx(&full[st], C::kStage);
                bulk_load_hint(stage, static_cast<const uint8_t *>(p.k_cache) + from, C::kTile, &full[st], policy);
                bulk_load_hint(stage + C::kTile, static_cast<const uint8_t *>(p.v_cache) + from, C::kTile, &full[st],
                               policy);
            }
        } else {  // a bad block id reads as zeros, as a block that nothing was written to
            for (int i = lane; i < C::kStage / 16; i += 32) reinterpret_cast<uint4 *>(stage)[i] = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();  // these writes before the copy that refills the stage
            __syncwarp();
            if (lane == 0) {
                raise_error(PKV_DEVERR_BLOCK_ID);
                mbar_arrive(&full[st]);
            }
        }
        ++issued;
    };
    while (issued < min(NS, cnt)) issue();

    const size_t slot_floats = (size_t)g * (2 + D);
    const __nv_bfloat16 *qbase = static_cast<const __nv_bfloat16 *>(p.q);
    WA wa;
    typename WA::QRaw raw;
    int seg_j0 = c.j, len = seq_len(p, c.s, false);
    WA::load_raw(raw, qbase + ((size_t)c.s * p.num_q_heads + (size_t)c.h * g) * D, g, lane);
    wa.set_q(raw, p.scale_log2, lane);
    wa.reset();
    E4m3Cut cut{0, w, 0, 0};
    int i = 0;
    bool waited = true;
    // N blocks from position i on, all of one unit
    auto step = [&](auto nb_tag, int valid) -> bool {
        constexpr int N = decltype(nb_tag)::value;
        uint32_t tile[N];
#pragma unroll
        for (int b = 0; b < N; ++b) {
            const int st = (i + b) & (NS - 1);
            if (!__all_sync(0xffffffffu, mbar_wait(&full[st], ((i + b) / NS) & 1))) return false;
            tile[b] = smem_u32(ring + st * C::kStage);
        }
        wa.template blocks<N>(tile, valid, lane);
        __syncwarp();  // every lane's reads of the stages are done before their refill
#pragma unroll
        for (int b = 0; b < N; ++b)
            if (issued < cnt) issue();
        return true;
    };
    while (true) {
        const bool two = NB == 2 && i + 1 < cnt && c.j + 1 < c.n;
        const int last_j = two ? c.j + 1 : c.j, last_i = two ? i + 1 : i;
        const bool unit_end = last_j == c.n - 1;
        Cursor cn = c;
        int len_next = 0;
        if (unit_end && last_i != cnt - 1) {  // the next unit's query and length, in flight while these blocks compute
            cn.j = last_j;
            cursor_advance(cn, 1, prefix, Hkv);
            WA::load_raw(raw, qbase + ((size_t)cn.s * p.num_q_heads + (size_t)cn.h * g) * D, g, lane);
            len_next = seq_len(p, cn.s, false);
        }
        const int valid = unit_end ? len - kBlock * (c.n - 1) : kBlock;  // tokens of the last of these blocks
        waited = two ? step(IntConst<NB>{}, valid) : step(IntConst<1>{}, valid);
        if (!waited) break;
        i = last_i;
        c.j = last_j;
        if (!unit_end && i != cnt - 1) {
            ++c.j;
            ++i;
            continue;
        }
        // ---- the segment ends here ----
        wa.reduce_l();
        const size_t orow = (size_t)c.s * p.num_q_heads + (size_t)c.h * g;
        if (seg_j0 == 0 && unit_end) {
            wa.store_rows(out + orow * D, g, lane);
        } else {
            // a cut unit: its state waits for the merge; the worker that holds its start records it
            wa.store_state(p.partials + (size_t)(2 * w + (seg_j0 == 0 ? 1 : 0)) * slot_floats, g, lane);
            if (seg_j0 == 0) {
                const long long x0 = (long long)Hkv * prefix[c.s] + (long long)c.h * c.n;
                cut.segments = (int)(((x0 + c.n) * W - 1) / T) - w + 1;
                cut.row = (int)orow;
            }
        }
        if (cuts_by_unit && seg_j0 == 0 && lane == 0) cuts[c.s * Hkv + c.h] = cut;
        if (i == cnt - 1) break;
        ++i;
        c = cn;
        seg_j0 = 0;
        len = len_next;
        wa.set_q(raw, p.scale_log2, lane);
        wa.reset();
    }
    if (!waited) {
        // a copy never landed: the output is unspecified; wait (bounded) for the others before leaving
        if (lane == 0) raise_error(PKV_DEVERR_TIMEOUT);
        const int left = cnt - i;
        for (; i < issued; ++i) mbar_wait(&full[i & (NS - 1)], (i / NS) & 1);
        // nothing of the units begun here and from here on is merged (their records hold what the workspace held)
        cut.segments = 0;
        if (cuts_by_unit && lane == 0) {
            if (seg_j0 == 0) cuts[c.s * Hkv + c.h] = cut;
            units_begun_later(
                c, left, [&](Cursor &at, int k) { cursor_advance(at, k, prefix, Hkv); },
                [&](int s, int h) { cuts[s * Hkv + h] = cut; });
        }
    }
    if (cuts && !cuts_by_unit && lane == 0) cuts[w] = cut;
}

// Merges the states of every cut unit: grid (records, head groups). A unit of a few segments is merged by a warp per
// query head; the warps of a CTA share longer ones, head by head, and join through shared memory. Either way
// eight segments' loads are in flight at a time; their latency is what the merge takes. Many units: four
// warps a record. Few units, of many segments each: sixteen warps a record and head.
template <int D, int NW, typename OutT>
__global__ void __launch_bounds__(NW * 32)
    e4m3_merge_kernel(OutT *out, const float *__restrict__ partials, const E4m3Cut *__restrict__ cuts, int g) {
    constexpr int PER = D / 32, NB = 8, kAlone = 16;  // segments one warp takes alone
    __shared__ float part[NW][2 + D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const E4m3Cut cut = cuts[blockIdx.x];
    const int nseg = cut.segments;
    if (nseg <= 0) return;
    float M, L, acc[PER];
    auto gather = [&](int head, int first, int step) {
        M = -INFINITY, L = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.f;
        for (int k0 = first; k0 < nseg; k0 += step * NB) {
            float m[NB], l[NB], o[NB][PER];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int k = k0 + b * step;
                m[b] = -INFINITY;
                l[b] = 0.f;
#pragma unroll
                for (int i = 0; i < PER; ++i) o[b][i] = 0.f;
                if (k < nseg) {  // the first segment ends its worker's range, the others begin theirs
                    const float *r =
                        partials + ((size_t)(2 * (cut.worker + k) + (k == 0 ? 1 : 0)) * g + head) * (2 + D);
                    m[b] = __ldcg(r);
                    l[b] = __ldcg(r + 1);
#pragma unroll
                    for (int i = 0; i < PER; ++i) o[b][i] = __ldcg(r + 2 + lane + 32 * i);
                }
            }
            float top = M;
#pragma unroll
            for (int b = 0; b < NB; ++b) top = fmaxf(top, m[b]);
            const float al = ex2_approx(M - top);
            M = top;
            L *= al;
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] *= al;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float f = ex2_approx(m[b] - top);
                L = fmaf(l[b], f, L);
#pragma unroll
                for (int i = 0; i < PER; ++i) acc[i] = fmaf(o[b][i], f, acc[i]);
            }
        }
    };
    if (nseg <= kAlone) {
        for (int head = blockIdx.y * NW + warp; head < g; head += gridDim.y * NW) {
            gather(head, 0, 1);
            const float inv = 1.f / L;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                out[(size_t)(cut.row + head) * D + lane + 32 * i] = to_out<OutT>(acc[i] * inv);
        }
        return;
    }
    for (int head = blockIdx.y; head < g; head += gridDim.y) {
        gather(head, warp, NW);
        if (lane == 0) {
            part[warp][0] = M;
            part[warp][1] = L;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) part[warp][2 + lane + 32 * i] = acc[i];
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += NW * 32) {  // (every warp saw a segment: nseg > kAlone >= NW)
            float top = -INFINITY;
            for (int v = 0; v < NW; ++v) top = fmaxf(top, part[v][0]);
            float sum = 0.f, o = 0.f;
            for (int v = 0; v < NW; ++v) {
                const float f = ex2_approx(part[v][0] - top);
                sum = fmaf(part[v][1], f, sum);
                o = fmaf(part[v][2 + d], f, o);
            }
            out[(size_t)(cut.row + head) * D + d] = to_out<OutT>(o / sum);
        }
        __syncthreads();
    }
}

}  // namespace pkv
