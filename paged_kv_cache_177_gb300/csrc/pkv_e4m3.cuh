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
// Decode over e4m3 tiles. The decomposition is the persistent bf16 kernel's: one CTA per SM,
// NW warps, each an independent worker with its own ring of NS stages; all (sequence, kv head)
// units' blocks form one line of T positions, cut into equal ranges, one per worker.
//
// The step over one staged (K, V) block, for the group's query heads as the MMA's N:
//   x_t = (scale log2 e) 2^(ek_t + eq) <codes K_t, q'>      q = q' 2^eq, q' in f16
//   y_t = x_t + ev_t;   m' = max(m, max_t y_t);   w_t = 2^(y_t - m')
//   l = l 2^(m - m') + sum_t 2^(x_t - m');   O = O 2^(m - m') + sum_t w_t codes V_t
// and the output is O / l. Codes widen to f16 without loss, and products with a query of 8
// significant bits are exact in the tensor cores' fp32 sums, so no code is multiplied by its scale:
// K's enters the score, V's the exponent of the weight. The reference m' follows y, not x, so the
// weights -- the one thing rounded here, to f16's 11 bits -- are largest where their values
// matter most, whatever the rows' scales. A row's exponent lies in [-50, 50], so sum 2^(x - m')
// neither overflows nor loses a term that counts.
//
// Codes come from shared memory by ldmatrix as pairs of bytes: a 16-byte chunk of a K row is the 16
// contraction elements of one MMA (4 t4 .. 4 t4 + 3 in lane t4: the order within a contraction
// is free as long as q's fragment has it too), and a transposed chunk of V holds two elements of
// two tokens a register, which one byte permutation sorts into the even and odd rows of O.
// =====================================================================================
template <int D, int NT>
struct WarpAttnE4m3 {
    static constexpr int kChunks = D / 16;  // 16-byte chunks of a row = MMAs of a block's QK^T, and of its PV
    using QRaw = uint2[kChunks][NT];        // q[head gq][16 c + 4 t4 .. + 3], bf16
    float m[NT][2], l[NT][2], qs[NT][2];    // of heads 2 t4, 2 t4 + 1 of each 8 columns; qs: score scale, log2 domain
    float acc[kChunks][NT][4];              // [.][.][e]: head 2 t4 + (e & 1), element 16 c + 2 gq + (e >> 1)
    uint32_t qf[kChunks][NT][2];

    // Shared address of 16-byte chunk c of row r: rows of D bytes under the D-byte TMA swizzle.
    static __device__ __forceinline__ uint32_t at(uint32_t tile, int r, int c) {
        return tile + r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
    }

    static __device__ __forceinline__ void load_raw(QRaw &raw, const __nv_bfloat16 *q_group, int g, int lane) {
        const int gq = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int hl = nt * 8 + gq;
            const __nv_bfloat16 *row = q_group + (size_t)(hl < g ? hl : 0) * D + 4 * t4;
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                raw[c][nt] = hl < g ? __ldg(reinterpret_cast<const uint2 *>(row + 16 * c)) : make_uint2(0u, 0u);
        }
    }

    // q to f16, each head scaled by a power of two that brings its largest element to [2^13, 2^14):
    // exact down to 2^-27 of that element.
    __device__ __forceinline__ void set_q(const QRaw &raw, float scale_log2, int lane) {
        const int t4 = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const uint32_t w[2] = {raw[c][nt].x, raw[c][nt].y};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float a = fabsf(__uint_as_float(w[i] << 16)), b = fabsf(__uint_as_float(w[i] & 0xffff0000u));
                    top = fmaxf(top, fmaxf(a < INFINITY ? a : 0.f, b < INFINITY ? b : 0.f));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // exponent of the scale, kept where both it and its reciprocal are normal numbers
            const int e = top > 0.f ? max(-100, min(113, (int)(__float_as_uint(top) >> 23) - 127 - 13)) : 0;
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const uint32_t w[2] = {raw[c][nt].x, raw[c][nt].y};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16) * inv,
                                                        __uint_as_float(w[i] & 0xffff0000u) * inv);
                    qf[c][nt][i] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
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
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[c][nt][e] = 0.f;
        }
    }

    // One staged block. Rows below lo are not tokens (the tile was loaded lo rows early and they are
    // zeros); kb, vb: scale bytes of this lane's two token rows gq and gq + 8.
    __device__ __forceinline__ void block(uint32_t sk, uint32_t sv, const uint32_t (&kb)[2], const uint32_t (&vb)[2],
                                          int lo, int lane) {
        const int gq = lane >> 2, mi = lane >> 3, r8 = lane & 7;
        const int row = r8 + (mi & 1) * 8;  // of this lane's ldmatrix addresses, K and V alike
        float sc[NT][4], sb[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nt][e] = sb[nt][e] = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; c += 2) {
            uint32_t k[4];
            ldsm_x4(at(sk, row, c + (mi >> 1)), k);
            const uint32_t a0[4] = {cvt_f16x2_e4m3x2(k[0]), cvt_f16x2_e4m3x2(k[1]), cvt_f16x2_e4m3x2(k[0] >> 16),
                                    cvt_f16x2_e4m3x2(k[1] >> 16)};
            const uint32_t a1[4] = {cvt_f16x2_e4m3x2(k[2]), cvt_f16x2_e4m3x2(k[3]), cvt_f16x2_e4m3x2(k[2] >> 16),
                                    cvt_f16x2_e4m3x2(k[3] >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_f16_16816(sc[nt], a0, qf[c][nt][0], qf[c][nt][1]);
                mma_f16_16816(sb[nt], a1, qf[c + 1][nt][0], qf[c + 1][nt][1]);
            }
        }
        const bool v0 = gq >= lo, v1 = gq + 8 >= lo;
        const float k0 = e8m0_value(kb[0]), k1 = e8m0_value(kb[1]);
        const float ev0 = (float)((int)vb[0] - 127), ev1 = (float)((int)vb[1] - 127);
        uint32_t p0[NT], p1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[4], y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool ok = e < 2 ? v0 : v1;
                x[e] = ok ? (sc[nt][e] + sb[nt][e]) * (e < 2 ? k0 : k1) * qs[nt][e & 1] : -INFINITY;
                y[e] = ok ? x[e] + (e < 2 ? ev0 : ev1) : -INFINITY;
            }
            float mx0 = fmaxf(y[0], y[2]), mx1 = fmaxf(y[1], y[3]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
            }
            const float mn0 = fmaxf(m[nt][0], mx0), mn1 = fmaxf(m[nt][1], mx1);  // finite: a block holds a token
            const float al0 = ex2_approx(m[nt][0] - mn0), al1 = ex2_approx(m[nt][1] - mn1);
            m[nt][0] = mn0;
            m[nt][1] = mn1;
            l[nt][0] = l[nt][0] * al0 + (ex2_approx(x[0] - mn0) + ex2_approx(x[2] - mn0));
            l[nt][1] = l[nt][1] * al1 + (ex2_approx(x[1] - mn1) + ex2_approx(x[3] - mn1));
            const __half2 w0 = __floats2half2_rn(ex2_approx(y[0] - mn0), ex2_approx(y[1] - mn1));
            const __half2 w1 = __floats2half2_rn(ex2_approx(y[2] - mn0), ex2_approx(y[3] - mn1));
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                acc[c][nt][0] *= al0;
                acc[c][nt][1] *= al1;
                acc[c][nt][2] *= al0;
                acc[c][nt][3] *= al1;
            }
            p0[nt] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&w0));
            p1[nt] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&w1));
        }
#pragma unroll
        for (int c = 0; c < kChunks; c += 2) {
            uint32_t v[4];
            ldsm_x4_trans(at(sv, row, c + (mi >> 1)), v);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __byte_perm(v[i], 0u, 0x3120);  // (t, d) (t + 1, d) | (t, d + 1) (t + 1, d + 1)
            const uint32_t a0[4] = {cvt_f16x2_e4m3x2(v[0]), cvt_f16x2_e4m3x2(v[0] >> 16), cvt_f16x2_e4m3x2(v[1]),
                                    cvt_f16x2_e4m3x2(v[1] >> 16)};
            const uint32_t a1[4] = {cvt_f16x2_e4m3x2(v[2]), cvt_f16x2_e4m3x2(v[2] >> 16), cvt_f16x2_e4m3x2(v[3]),
                                    cvt_f16x2_e4m3x2(v[3] >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_f16_16816(acc[c][nt], a0, p0[nt], p1[nt]);
                mma_f16_16816(acc[c + 1][nt], a1, p0[nt], p1[nt]);
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
                for (int c = 0; c < kChunks; ++c) {
                    OutT *o = rows + (size_t)head * D + 16 * c + 2 * gq;
                    o[0] = to_out<OutT>(acc[c][nt][e] * inv);
                    o[1] = to_out<OutT>(acc[c][nt][e + 2] * inv);
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
                for (int c = 0; c < kChunks; ++c)
                    *reinterpret_cast<float2 *>(row + 2 + 16 * c + 2 * gq) = make_float2(acc[c][nt][e], acc[c][nt][e + 2]);
            }
    }
};

template <int D, int NS, int NW>
struct E4m3Cfg {
    static constexpr int kTile = kBlock * D;  // codes of one (block, head) tile
    static constexpr int kStage = 2 * kTile;  // K, then V
    static constexpr int kThreads = NW * 32;
    static constexpr int kScaleOff = NW * NS * kStage;               // [NW][NS] x (16 K, 16 V scale bytes)
    static constexpr int kBarOff = kScaleOff + NW * NS * 2 * kBlock;
    static constexpr int kPrefixOff = kBarOff + NW * NS * 8;
    static constexpr size_t smem_bytes(int num_seqs) { return kPrefixOff + (size_t)(num_seqs + 1) * 4 + 1024; }
    static_assert((NS & (NS - 1)) == 0 && NS <= 32, "stage index and bad-block bits");
};

// A unit cut by the end of worker w's range, begun in it: its segments (0: none) and first output row.
struct E4m3Cut {
    int segments, row;
};

template <int D, int NT, int NS, int NW, typename OutT>
__global__ void __launch_bounds__(NW * 32, 1)
    decode_e4m3_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                       const DecodeParams p, E4m3Cut *cuts, const int whole_units) {
    using C = E4m3Cfg<D, NS, NW>;
    using WA = WarpAttnE4m3<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int warp_total[NW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.num_seqs, Hkv = p.num_kv_heads, g = p.group;
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(base + C::kBarOff) + warp * NS;
    int *prefix = reinterpret_cast<int *>(base + C::kPrefixOff);
    OutT *out = static_cast<OutT *>(p.out);
    if (tid == 0) {
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
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
        }

    // this worker's range of positions: an equal share, or (short contexts) a share of whole units
    const long long T = (long long)Hkv * prefix[S];
    const int all = gridDim.x * NW, w = blockIdx.x * NW + warp;
    const long long U = (long long)S * Hkv;
    const int W = (int)min((long long)all, whole_units ? U : max(1LL, T / 2));
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
        if (cuts && lane == 0) cuts[w].segments = 0;
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
    // each with 16 * kv head + the rows its tile is loaded early.
    struct Batch {
        int pb, hs;
    };
    auto batch_of = [&](Cursor b, int count) -> Batch {
        Batch r{0, 0};
        if (lane < count) {
            cursor_advance(b, lane, prefix, Hkv);
            r.pb = __ldg(p.block_tables + (size_t)b.s * p.max_blocks_per_seq + b.j);
            r.hs = b.h * 16 + ((b.j == b.n - 1) ? kBlock * b.n - seq_len(p, b.s, false) : 0);
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
    uint8_t *scales = base + C::kScaleOff + warp * NS * 2 * kBlock;
    const uint64_t policy = l2_evict_first();
    int issued = 0;
    uint32_t bad = 0;  // bit of a stage whose block id is out of range: it reads as zeros
    auto issue = [&]() {
        if (issued > 0 && (issued & 31) == 0) {
            cur = nxt;
            if (issued + 32 < cnt) {
                cursor_advance(bnext, 32, prefix, Hkv);
                nxt = batch_of(bnext, min(32, cnt - issued - 32));
            }
        }
        const int pb = __shfl_sync(0xffffffffu, cur.pb, issued & 31);
        const int hs = __shfl_sync(0xffffffffu, cur.hs, issued & 31);
        const int st = issued & (NS - 1);
        const bool ok = pb >= 0 && pb < p.num_blocks;
        bad = (bad & ~(1u << st)) | ((ok ? 0u : 1u) << st);
        if (lane == 0) {
            if (!ok) raise_error(PKV_DEVERR_BLOCK_ID);
            const int z = ok ? pb * Hkv + (hs >> 4) : -1, y = -(hs & 15);
            mbar_arrive_expect_tx(&full[st], C::kStage + (ok ? 2 * kBlock : 0));
            tma_load_3d_hint(ring + st * C::kStage, &tmk, 0, y, z, &full[st], policy);
            tma_load_3d_hint(ring + st * C::kStage + C::kTile, &tmv, 0, y, z, &full[st], policy);
            if (ok) {
                const size_t tail = (size_t)z * PKV_E4M3_TILE_BYTES(D) + kBlock * D;
                bulk_load(scales + st * 2 * kBlock, static_cast<const uint8_t *>(p.k_cache) + tail, kBlock, &full[st]);
                bulk_load(scales + st * 2 * kBlock + kBlock, static_cast<const uint8_t *>(p.v_cache) + tail, kBlock,
                          &full[st]);
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
    E4m3Cut cut{0, 0};
    int i = 0;
    bool waited = true;
    for (; i < cnt; ++i) {
        const int st = i & (NS - 1);
        const bool unit_end = c.j == c.n - 1;
        Cursor cn = c;
        int len_next = 0;
        if (unit_end && i != cnt - 1) {  // the next unit's query and length, in flight while this block computes
            cursor_advance(cn, 1, prefix, Hkv);
            WA::load_raw(raw, qbase + ((size_t)cn.s * p.num_q_heads + (size_t)cn.h * g) * D, g, lane);
            len_next = seq_len(p, cn.s, false);
        }
        if (!(waited = __all_sync(0xffffffffu, mbar_wait(&full[st], (i / NS) & 1)))) break;
        const int lo = unit_end ? kBlock * c.n - len : 0;
        const uint8_t *sb = scales + st * 2 * kBlock;
        const int r0 = max((lane >> 2) - lo, 0), r1 = max((lane >> 2) + 8 - lo, 0);
        const bool isbad = (bad >> st) & 1;
        const uint32_t kb[2] = {isbad ? 127u : sb[r0], isbad ? 127u : sb[r1]};
        const uint32_t vb[2] = {isbad ? 127u : sb[kBlock + r0], isbad ? 127u : sb[kBlock + r1]};
        const uint32_t sk = smem_u32(ring + st * C::kStage);
        wa.block(sk, sk + C::kTile, kb, vb, lo, lane);
        __syncwarp();  // every lane's reads of the stage are done before its refill
        if (issued < cnt) issue();
        if (!unit_end && i != cnt - 1) {
            ++c.j;
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
        if (i == cnt - 1) break;
        c = cn;
        seg_j0 = 0;
        len = len_next;
        wa.set_q(raw, p.scale_log2, lane);
        wa.reset();
    }
    if (!waited) {
        // a copy never landed: the output is unspecified; wait (bounded) for the others before leaving
        if (lane == 0) raise_error(PKV_DEVERR_TIMEOUT);
        for (++i; i < issued; ++i) mbar_wait(&full[i & (NS - 1)], (i / NS) & 1);
        cut.segments = 0;
    }
    if (cuts && lane == 0) cuts[w] = cut;
}

// Merges the states of every cut unit: one CTA per worker that began one. Up to 64 segments a warp
// takes whole heads (the segments' loads overlap); more are shared among the warps head by head.
template <int D, typename OutT>
__global__ void __launch_bounds__(256)
    e4m3_merge_kernel(OutT *out, const float *__restrict__ partials, const E4m3Cut *__restrict__ cuts, int g) {
    constexpr int PER = D / 32;
    __shared__ float part[8][2 + D];
    const int w1 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const E4m3Cut cut = cuts[w1];
    const int nseg = cut.segments;
    if (nseg <= 0) return;
    auto row_of = [&](int k, int head) {
        return partials + ((size_t)(2 * (w1 + k) + (k == 0 ? 1 : 0)) * g + head) * (2 + D);
    };
    // segments first, first + step, ...: their max, weight sum and weighted outputs
    auto gather = [&](int head, int first, int step, float &M, float &L, float (&acc)[PER]) {
        M = -INFINITY;
        for (int k = first + lane * step; k < nseg; k += 32 * step) M = fmaxf(M, row_of(k, head)[0]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        L = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 4
        for (int k = first; k < nseg; k += step) {
            const float *r = row_of(k, head);
            const float f = ex2_approx(r[0] - M);
            L = fmaf(r[1], f, L);
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] = fmaf(r[2 + lane + 32 * i], f, acc[i]);
        }
    };
    float M, L, acc[PER];
    if (nseg <= 64) {
        for (int head = warp; head < g; head += 8) {
            gather(head, 0, 1, M, L, acc);
            const float inv = 1.f / L;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                out[(size_t)(cut.row + head) * D + lane + 32 * i] = to_out<OutT>(acc[i] * inv);
        }
        return;
    }
    for (int head = 0; head < g; ++head) {
        gather(head, warp, 8, M, L, acc);
        if (lane == 0) {
            part[warp][0] = M;
            part[warp][1] = L;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) part[warp][2 + lane + 32 * i] = acc[i];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int v = 0; v < 8; ++v) M = fmaxf(M, part[v][0]);
            L = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const float f = ex2_approx(part[v][0] - M);
                L = fmaf(part[v][1], f, L);
#pragma unroll
                for (int i = 0; i < PER; ++i) acc[i] = fmaf(part[v][2 + lane + 32 * i], f, acc[i]);
            }
            const float inv = 1.f / L;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                out[(size_t)(cut.row + head) * D + lane + 32 * i] = to_out<OutT>(acc[i] * inv);
        }
        __syncthreads();
    }
}

}  // namespace pkv
