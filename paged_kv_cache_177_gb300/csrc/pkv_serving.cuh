// pkv_serving.cuh -- host side of the serving calls around the cache: the
// 8-bit cache, the pass from the projections to the cache, trees of drafted
// tokens and their verification, transformed scores, and prefixes shared by
// many sequences. Included by pkv.cu, whose helpers it uses.
#pragma once

namespace {

// Whether two stretches of memory share a byte.
bool overlaps(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

// Arguments that every call over [num_blocks][num_kv_heads] tiles shares.
int check_pool(int num_kv_heads, int num_blocks, int head_dim) {
    if (num_kv_heads <= 0 || num_blocks <= 0) return PKV_ERR_ARG;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)num_blocks * num_kv_heads * 16 >= (int64_t(1) << 31)) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// The arguments that the attention calls share, into p.
int attention_params(pkv::DecodeParams &p, void *out, const void *q, const void *k_cache, const void *v_cache,
                     const int32_t *block_tables, const int32_t *context_lens, float scale, int num_kv_heads,
                     int num_seqs, int num_q_heads, int head_dim, int max_blocks_per_seq, int num_blocks,
                     int max_context_len, int max_group) {
    if (num_seqs < 0 || num_kv_heads <= 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        max_context_len < 0)
        return PKV_ERR_ARG;
    int rc;
    if ((rc = check_pool(num_kv_heads, num_blocks, head_dim)) != PKV_OK) return rc;
    if (num_q_heads % num_kv_heads != 0) return PKV_ERR_ARG;
    if (num_q_heads / num_kv_heads > max_group) return PKV_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return PKV_ERR_ARG;
    if (num_seqs > 65535) return PKV_ERR_UNSUPPORTED;
    if (max_blocks_per_seq > INT32_MAX / 16) return PKV_ERR_UNSUPPORTED;
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.max_context_len = max_context_len;
    return PKV_OK;
}

template <typename T>
int launch_append_e4m3(const void *k, const void *v, const int64_t *slots, void *kc, void *vc, int num_tokens,
                       int num_kv_heads, int head_dim, int num_blocks, cudaStream_t st) {
    const int per = pkv::kAppendThreads / (head_dim / 8);  // tokens of a CTA
    auto kern = head_dim == 128 ? pkv::kv_append_e4m3_kernel<T, 128> : pkv::kv_append_e4m3_kernel<T, 64>;
    kern<<<dim3((num_tokens + per - 1) / per, num_kv_heads), pkv::kAppendThreads, 0, st>>>(
        static_cast<const T *>(k), static_cast<const T *>(v), slots, static_cast<uint8_t *>(kc),
        static_cast<uint8_t *>(vc), num_tokens, num_kv_heads, num_blocks);
    return check_launch();
}

template <typename T>
int launch_dequantize(void *dk, void *dv, int dst_nb, const void *sk, const void *sv, int src_nb,
                      const int64_t *pairs, int num_pairs, int num_kv_heads, int head_dim, cudaStream_t st) {
    auto kern = head_dim == 128 ? pkv::dequantize_blocks_kernel<T, 128> : pkv::dequantize_blocks_kernel<T, 64>;
    const dim3 grid((num_kv_heads * head_dim + pkv::kReadBackThreads - 1) / pkv::kReadBackThreads,
                    num_pairs < 65535 ? num_pairs : 65535, 2);
    kern<<<grid, pkv::kReadBackThreads, 0, st>>>(static_cast<T *>(dk), static_cast<T *>(dv),
                                                 static_cast<const uint8_t *>(sk), static_cast<const uint8_t *>(sv),
                                                 pairs, num_pairs, num_kv_heads, src_nb, dst_nb);
    return check_launch();
}

// Decode over e4m3 tiles: the persistent kernel's warps, each a worker with its ring. A worker's step is one chain of
// dependent instructions, so as many run as their registers allow without spilling: twelve at head_dim 128 and
// sixteen at 64 with up to 8 heads to a kv head, eight and twelve with more, whose accumulators are twice as many.
// head_dim 128, 256 contexts around 1000, 32 q / 8 kv heads: 119 us, 132 with ten, 142 with eight; 64: 128 such contexts
// 39.6 us, 43.4 with twelve, 40.6 with twenty. 16 heads to a kv head, 8 kv heads, 256 contexts around 1000, head_dim 128: 175 us,
// 222 with six, 223 with ten (64 contexts of 2 kv heads, which make few states: 29, 26, 34); head_dim 64, 256 contexts
// of 1000-2000: 112 us, 138 with ten.
constexpr int e4m3_warps(int head_dim, int group) { return head_dim == 128 ? (group <= 8 ? 12 : 8) : (group <= 8 ? 16 : 12); }
constexpr int kE4m3MaxSeqs = 4096;  // sequences of one launch: their block counts lie in shared memory

// Contexts this short are not cut: a worker takes whole (sequence, kv head) units and writes
// their outputs itself, so no merge is launched. (32 q / 8 kv heads, whole and cut: 4 contexts of up to 64 tokens
// 8.5 and 12.2 us, of up to 96 12.0 and 11.5; 64 of up to 96 12.3 and 12.7, of up to 128 14.4 and 12.8, of up to
// 256 22.8 and 14.0; 1000 of up to 64 32.6 and 34.6, of up to 128 51.9 and 48.3.)
bool e4m3_whole_units(int max_context_len) { return max_context_len <= 96; }

template <int D, int NT, typename OutT>
int launch_decode_e4m3_shape(pkv::DecodeParams &p, void *workspace, cudaStream_t st) {
    // Four stages of a block's K and V: 16 KB a warp at head_dim 128, where a step takes one block, whose stage is
    // refilled at once (32K-128K contexts, merge left out: 234 us, and 249 us with two blocks a step, whose stages
    // wait for each other); at 64 a step of two blocks hides its latencies better than it costs (128
    // contexts around 1000: 40 us, 44 with one).
    constexpr int NW = e4m3_warps(D, 8 * NT), NS = 4, NB = D == 128 ? 1 : 2;
    using C = pkv::E4m3Cfg<D, NS, NW>;
    static_assert(C::smem_bytes(kE4m3MaxSeqs) + 64 <= kSmemLimit, "shared memory");
    auto kern = pkv::decode_e4m3_kernel<D, NT, NB, NS, NW, OutT>;
    static thread_local int configured_device = -1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    if (configured_device != dev) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)C::smem_bytes(kE4m3MaxSeqs)) != cudaSuccess)
            return PKV_ERR_CUDA;
        configured_device = dev;
    }
    int sms = 0;
    if (sm_count(&sms) != PKV_OK) return PKV_ERR_CUDA;
    const int grid = sms < kPersistMaxCtas ? sms : kPersistMaxCtas;
    const bool whole = e4m3_whole_units(p.max_context_len);
    pkv::E4m3Cut *cuts = nullptr;
    if (!whole) {
        cuts = reinterpret_cast<pkv::E4m3Cut *>(static_cast<char *>(workspace) + kCounterBytes);
        p.partials = reinterpret_cast<float *>(cuts + (size_t)kPersistMaxCtas * NW);
    }
    const long long units = (long long)p.num_seqs * p.num_kv_heads;
    const bool by_unit = !whole && units <= grid * NW;
    kern<<<grid, C::kThreads, C::smem_bytes(p.num_seqs), st>>>(p, cuts, whole ? 1 : 0, by_unit ? 1 : 0);
    const int rc = check_launch();
    if (rc != PKV_OK || whole) return rc;
    // (80 units of 8000 tokens: 37.3 us with the wide merge, 40.5 with the narrow one; 224 of 4000: 47.1, 45.8; 512: 95, 89)
    const bool few = by_unit && 8 * units <= grid * NW;
    auto merge = [&](auto kernel, int warps) {
        return launch_pdl(kernel, dim3(by_unit ? (unsigned)units : grid * NW, few ? p.group : (p.group + 3) / 4),
                          dim3(warps * 32), 0, st, static_cast<OutT *>(p.out), static_cast<const float *>(p.partials),
                          static_cast<const pkv::E4m3Cut *>(cuts), p.group);
    };
    return few ? merge(pkv::e4m3_merge_kernel<D, 16, OutT>, 16) : merge(pkv::e4m3_merge_kernel<D, 4, OutT>, 4);
}

template <typename OutT>
int launch_decode_e4m3(pkv::DecodeParams &p, int head_dim, void *workspace, cudaStream_t st) {
    if (head_dim == 128)
        return p.group <= 8 ? launch_decode_e4m3_shape<128, 1, OutT>(p, workspace, st)
                            : launch_decode_e4m3_shape<128, 2, OutT>(p, workspace, st);
    return p.group <= 8 ? launch_decode_e4m3_shape<64, 1, OutT>(p, workspace, st)
                        : launch_decode_e4m3_shape<64, 2, OutT>(p, workspace, st);
}

// Trees: contexts of at most four chunks of 128 keys are not cut, so no merge is launched. (16 drafts, 32 q / 8 kv heads,
// whole and cut: 4 contexts of 240-480 tokens 13.2 and 15.7 us, of 450-900 18.0 and 16.6; 64: 35.0 and 35.4, 47.6 and 45.2.)
bool tree_whole_units(int max_context_len) { return max_context_len <= 512; }

// Two row tiles to a unit where one does not hold the largest tree's rows.
bool tree_pair(int g, int max_query_len) { return max_query_len > 128 / g; }

template <int D, bool kPair, bool kPrefix = false>
int launch_tree(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv, const pkv::TreeParams &tp,
                int q_tokens, void *workspace, cudaStream_t st) {
    using C = pkv::TreeCfg<D, kPair>;
    static_assert(C::kSmem <= (int)kSmemLimit, "shared memory");
    auto kern = pkv::tree_attention_kernel<D, kPair, kPrefix>;
    static thread_local int configured_device = -1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    if (configured_device != dev) {
        // the register split draws on the registers the CTA is launched with
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return PKV_ERR_CUDA;
        if (fa.numRegs * C::kThreads < 128 * C::kLowRegs + 256 * C::kHighRegs) return PKV_ERR_UNSUPPORTED;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
            return PKV_ERR_CUDA;
        configured_device = dev;
    }
    int sms = 0;
    if (sm_count(&sms) != PKV_OK) return PKV_ERR_CUDA;
    const int grid = sms < kPersistMaxCtas ? sms : kPersistMaxCtas, g = tp.d.group, tile_tokens = 128 / g;
    const bool whole = tree_whole_units(tp.d.max_context_len);
    pkv::TreeCut *cuts = nullptr;
    float *partials = nullptr;
    if (!whole) {
        cuts = reinterpret_cast<pkv::TreeCut *>(static_cast<char *>(workspace) + kCounterBytes);
        partials = reinterpret_cast<float *>(cuts + kPersistMaxCtas);
    }
    int rc;
    if constexpr (kPrefix) {  // (its set-up beside the plan, for which it waits)
        rc = launch_pdl(kern, dim3(grid), dim3(C::kThreads), C::kSmem, st, tmq, tmk, tmv, tp, partials, cuts, tile_tokens,
                        q_tokens);
    } else {
        kern<<<grid, C::kThreads, C::kSmem, st>>>(tmq, tmk, tmv, tp, partials, cuts, tile_tokens, q_tokens);
        rc = check_launch();
    }
    if (rc != PKV_OK || whole) return rc;
    const int per_set = C::kTiles * tile_tokens;
    const int rows = (tp.max_query_len < per_set ? tp.max_query_len : per_set) * g;  // of the largest unit
    return launch_pdl(pkv::tree_merge_kernel<D, kPrefix>, dim3(grid, (rows + 7) / 8), dim3(256), 0, st,
                      static_cast<__nv_bfloat16 *>(tp.d.out), tp.prefix_ml, tp.prefix_o, static_cast<const float *>(partials),
                      static_cast<const pkv::TreeCut *>(cuts), C::kUnitRows, g, tp.d.num_q_heads, tile_tokens);
}

// Warps an SM that few tokens are spread over. (Tokens of 48 heads of 128, bf16: 256 take 6.1 us, 5.8 with 12 warps and 8.4
// with 48; 700 take 7.8, 8.0 and 10.3; 1500 take 9.8, 11.1 and 13.0; 64 and fewer are the launch either way.)
constexpr int kRopeWarpsPerSm = 24;

template <typename T, int D>
int launch_rope(pkv::RopeParams p, bool interleaved, bool e4m3, cudaStream_t st) {
    auto kern = interleaved ? (e4m3 ? pkv::qk_norm_rope_append_kernel<T, D, true, true>
                                    : pkv::qk_norm_rope_append_kernel<T, D, true, false>)
                            : (e4m3 ? pkv::qk_norm_rope_append_kernel<T, D, false, true>
                                    : pkv::qk_norm_rope_append_kernel<T, D, false, false>);
    // warps to a token: as many as its rows can use while there are few tokens, one where tokens alone fill
    // the SMs' warps
    constexpr int rows_per_warp = 256 / D;
    const int passes = (p.num_q_heads + 2 * p.num_kv_heads + rows_per_warp - 1) / rows_per_warp;
    int sms = 0;
    if (sm_count(&sms) != PKV_OK) return PKV_ERR_CUDA;
    const int want = (int)((long long)sms * kRopeWarpsPerSm / p.num_tokens);
    p.warps_per_token = want < 1 ? 1 : want > passes ? passes : want;
    const long long blocks = ((long long)p.num_tokens * p.warps_per_token + pkv::kRopeWarps - 1) / pkv::kRopeWarps;
    kern<<<(unsigned)blocks, pkv::kRopeWarps * 32, 0, st>>>(p);
    return check_launch();
}

// CTAs of the cluster that takes a pair of query tiles: pairs, of which there are so many at most, each over `chunks` chunks
// at most; resident[i]: clusters of 2^i CTAs that the card holds. A round of clusters is taken to last as long as the
// chunks of one of its CTAs and eight more; up to three chunks, joining costs more than it saves.
// (With one, two, four and eight, 32 q / 8 kv heads of 128, capped: 16 tokens behind 16K 333, 173, 93, 53 us, behind 1K 27,
// 18, 14, 13; 512 behind 8K 197, 110, 124, 199; 8 x 64 behind 1K 34, 27, 43, 95, behind 4K 105, 63, 79, 142; 24 x 64 behind 4K
// 208, 183, 228, 371; 18 x 64 107, 124, 156, 285; prompts of 256 13.4, 15.0, 14.9, 41, of 512 20, 19, 30, 71, of
// 768 26, 32, 48, 105. The card holds 76, 36 and 15 clusters of two, four and eight.)
// These are batches of equal lengths. One width serves a launch, so a batch of mixed ones counts as all as long as its longest:
// 16 tokens behind 16K take 50 us alone, forty sequences of 4 behind 500 47, and both in one call 173, in clusters of two.
int prefill_scored_ctas(long long pairs, long long chunks, const int (&resident)[4]) {
    int best = 0;
    long long least = 0;
    for (int i = 0; i < (chunks > 3 ? 4 : 1) && resident[i] > 0; ++i) {
        const long long c = 1 << i, rounds = (pairs + resident[i] - 1) / resident[i];
        const long long cost = rounds * ((chunks + c - 1) / c + 8);
        if (i == 0 || cost < least) {
            best = i;
            least = cost;
        }
    }
    return 1 << best;
}

template <int D, bool kCap, bool kBias>
int launch_prefill_scored(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                          pkv::ScoredPrefillParams sp, dim3 grid, long long pairs, long long chunks, cudaStream_t st) {
    using C = pkv::TcCfg<D>;
    static_assert(C::kSmem <= (int)kSmemLimit, "shared memory");
    auto kern = pkv::prefill_scored_kernel<D, kCap, kBias>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static thread_local int configured_device = -1;
    static thread_local int resident[4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    if (configured_device != dev) {
        // the register split draws on the registers the CTA is launched with
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return PKV_ERR_CUDA;
        if (fa.numRegs * C::kThreads < 128 * C::kLowRegs + C::kTiles * 128 * C::kHighRegs) return PKV_ERR_UNSUPPORTED;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
            return PKV_ERR_CUDA;
        if (sm_count(&resident[0]) != PKV_OK) return PKV_ERR_CUDA;
        for (int i = 1; i < 4; ++i) {
            attr[0].val.clusterDim.x = 1 << i;
            cfg.gridDim = dim3(1 << i);
            if (cudaOccupancyMaxActiveClusters(&resident[i], kern, &cfg) != cudaSuccess) return PKV_ERR_CUDA;
        }
        configured_device = dev;
    }
    sp.ctas = prefill_scored_ctas(pairs, chunks, resident);
    if (sp.ctas == 1) {
        kern<<<grid, C::kThreads, C::kSmem, st>>>(tmq, tmk, tmv, sp);
        return check_launch();
    }
    grid.x *= sp.ctas;
    cfg.gridDim = grid;
    cfg.stream = st;
    attr[0].val.clusterDim.x = sp.ctas;
    return cudaLaunchKernelEx(&cfg, kern, tmq, tmk, tmv, sp) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int D>
int launch_prefill_scored(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                          const pkv::ScoredPrefillParams &sp, dim3 grid, long long pairs, long long chunks,
                          cudaStream_t st) {
    const bool bias = sp.pp.d.slopes != nullptr;
    if (sp.pp.d.cap_log2 != 0.f)
        return bias ? launch_prefill_scored<D, true, true>(tmq, tmk, tmv, sp, grid, pairs, chunks, st)
                    : launch_prefill_scored<D, true, false>(tmq, tmk, tmv, sp, grid, pairs, chunks, st);
    return bias ? launch_prefill_scored<D, false, true>(tmq, tmk, tmv, sp, grid, pairs, chunks, st)
                : launch_prefill_scored<D, false, false>(tmq, tmk, tmv, sp, grid, pairs, chunks, st);
}

// CTAs of the cluster that takes a sequence. Few sequences share their rows among up to eight CTAs, as long as all fit
// the card at once (two an SM) and a CTA's warps have a step each; large rows are shared anyway, down to 512 KB of p a CTA, or
// 128 KB each of p and q, which are read again for every further refusal while other sequences are done.
// (With one, two, four and eight: trees of up to six drafts over 131072 tokens, fp32, 16 sequences 42, 27, 20, 16 us; 64 47,
// 32, 27, 26; 128 60, 48, 41, 48; 256 79, 63, 60, 78; over 32000 64 21, 17, 17, 21, 256 30, 30, 41, 69; without q, over
// 131072, 16 17, 13, 11, 11, 64 20, 16, 15, 22; 256 38, 40, 46, 69.)
int verify_ctas(int num_seqs, int vocab, int elem, bool draft, int sms) {
    const int64_t weight = (int64_t)vocab * elem * (draft ? 4 : 1);
    int c = 8;
    while (c > 1 && (((long long)num_seqs * c > 2LL * sms && weight < (int64_t)c << 19) || vocab < 2048LL * c)) c /= 2;
    return c;
}

template <typename T>
int launch_verify(const pkv::VerifyParams &p, int num_seqs, cudaStream_t st) {
    int sms = 0;
    if (sm_count(&sms) != PKV_OK) return PKV_ERR_CUDA;
    const int c = verify_ctas(num_seqs, p.vocab, sizeof(T), p.draft != nullptr, sms);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)num_seqs * c);
    cfg.blockDim = dim3(pkv::kVerifyThreads);
    cfg.dynamicSmemBytes = sizeof(pkv::VerifyShared);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pkv::verify_drafts_kernel<T>, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

extern "C" {

int kv_append_e4m3(const void *k, const void *v, const int64_t *slot_mapping, void *k_cache, void *v_cache,
                   int num_tokens, int num_kv_heads, int head_dim, int num_blocks, pkv_dtype dtype, void *stream) {
    if (num_tokens < 0) return PKV_ERR_ARG;
    int rc;
    if ((rc = check_pool(num_kv_heads, num_blocks, head_dim)) != PKV_OK) return rc;
    if (!dtype_ok(dtype)) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PKV_BF16 ? launch_append_e4m3<__nv_bfloat16>(k, v, slot_mapping, k_cache, v_cache, num_tokens,
                                                                 num_kv_heads, head_dim, num_blocks, st)
                             : launch_append_e4m3<float>(k, v, slot_mapping, k_cache, v_cache, num_tokens,
                                                         num_kv_heads, head_dim, num_blocks, st);
}

int dequantize_blocks(void *dst_k_cache, void *dst_v_cache, int dst_num_blocks, const void *src_k_cache,
                      const void *src_v_cache, int src_num_blocks, const int64_t *src_dst_pairs, int num_pairs,
                      int num_kv_heads, int head_dim, pkv_dtype dst_dtype, void *stream) {
    if (num_pairs < 0 || dst_num_blocks <= 0) return PKV_ERR_ARG;
    int rc;
    if ((rc = check_pool(num_kv_heads, src_num_blocks, head_dim)) != PKV_OK) return rc;
    if ((rc = check_pool(num_kv_heads, dst_num_blocks, head_dim)) != PKV_OK) return rc;
    if (!dtype_ok(dst_dtype)) return PKV_ERR_UNSUPPORTED;
    if (num_pairs == 0) return PKV_OK;
    if (!dst_k_cache || !dst_v_cache || !src_k_cache || !src_v_cache || !src_dst_pairs) return PKV_ERR_ARG;
    if (!aligned16(dst_k_cache) || !aligned16(dst_v_cache) || !aligned16(src_k_cache) || !aligned16(src_v_cache))
        return PKV_ERR_ALIGN;
    const size_t dst_bytes = (size_t)dst_num_blocks * num_kv_heads * tile_vecs(dst_dtype, head_dim) * 16;
    const size_t src_bytes = (size_t)src_num_blocks * num_kv_heads * tile_vecs(PKV_E4M3, head_dim) * 16;
    for (const void *dst : {dst_k_cache, dst_v_cache})
        for (const void *src : {src_k_cache, src_v_cache})
            if (overlaps(dst, dst_bytes, src, src_bytes)) return PKV_ERR_OVERLAP;
    if (overlaps(dst_k_cache, dst_bytes, dst_v_cache, dst_bytes)) return PKV_ERR_OVERLAP;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dst_dtype == PKV_BF16
               ? launch_dequantize<__nv_bfloat16>(dst_k_cache, dst_v_cache, dst_num_blocks, src_k_cache, src_v_cache,
                                                  src_num_blocks, src_dst_pairs, num_pairs, num_kv_heads, head_dim, st)
               : launch_dequantize<float>(dst_k_cache, dst_v_cache, dst_num_blocks, src_k_cache, src_v_cache,
                                          src_num_blocks, src_dst_pairs, num_pairs, num_kv_heads, head_dim, st);
}

size_t pkv_e4m3_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_context_len) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_q_heads % num_kv_heads != 0 ||
        e4m3_whole_units(max_context_len))
        return 0;
    const size_t workers = (size_t)kPersistMaxCtas * e4m3_warps(head_dim, num_q_heads / num_kv_heads);
    return kCounterBytes + workers * sizeof(pkv::E4m3Cut) +
           workers * 2 * (num_q_heads / num_kv_heads) * (2 + (size_t)head_dim) * sizeof(float);
}

int paged_decode_attention_e4m3(void *out, const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *block_tables, const int32_t *context_lens, float scale,
                                int num_kv_heads, int num_seqs, int num_q_heads, int head_dim, int max_blocks_per_seq,
                                int num_blocks, int max_context_len, pkv_dtype dtype, void *workspace,
                                size_t workspace_bytes, void *stream) {
    pkv::DecodeParams p{};
    int rc;
    if ((rc = attention_params(p, out, q, k_cache, v_cache, block_tables, context_lens, scale, num_kv_heads, num_seqs,
                               num_q_heads, head_dim, max_blocks_per_seq, num_blocks, max_context_len, 16)) != PKV_OK)
        return rc;
    if (dtype != PKV_BF16 && dtype != PKV_BF16_OUT_F32) return PKV_ERR_UNSUPPORTED;
    // the kernel counts a launch's blocks, and a sequence's over its kv heads, in 32 bits
    const int64_t long_blocks = std::min<int64_t>(((int64_t)max_context_len + 15) / 16, max_blocks_per_seq);
    if (long_blocks * std::max(num_kv_heads, std::min(num_seqs, kE4m3MaxSeqs)) > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PKV_ERR_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ALIGN;
    const size_t need = pkv_e4m3_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return PKV_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // the kernel keeps the batch's block counts in shared memory: larger batches go in slices
    for (int s0 = 0; s0 < num_seqs; s0 += kE4m3MaxSeqs) {
        pkv::DecodeParams ps = p;
        const size_t row = (size_t)s0 * num_q_heads * head_dim;
        ps.out = static_cast<char *>(out) + row * (dtype == PKV_BF16 ? 2 : 4);
        ps.q = static_cast<const char *>(q) + row * 2;
        ps.block_tables = block_tables + (size_t)s0 * max_blocks_per_seq;
        ps.context_lens = context_lens + s0;
        ps.num_seqs = num_seqs - s0 < kE4m3MaxSeqs ? num_seqs - s0 : kE4m3MaxSeqs;
        rc = dtype == PKV_BF16 ? launch_decode_e4m3<__nv_bfloat16>(ps, head_dim, workspace, st)
                               : launch_decode_e4m3<float>(ps, head_dim, workspace, st);
        if (rc != PKV_OK) return rc;
    }
    return PKV_OK;
}

int qk_norm_rope_append(void *q_out, const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                        int64_t v_stride, const void *q_weight, const void *k_weight, float eps,
                        const int64_t *positions, int num_axes, const float *inv_freq, const int32_t *axes,
                        int rot_dim, int interleaved, const int64_t *slot_mapping, void *k_cache, void *v_cache,
                        int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                        pkv_dtype dtype, pkv_dtype cache_dtype, void *stream) {
    if (num_tokens < 0 || num_q_heads <= 0 || rot_dim < 0) return PKV_ERR_ARG;
    int rc;
    if ((rc = check_pool(num_kv_heads, num_blocks, head_dim)) != PKV_OK) return rc;
    if (!dtype_ok(dtype) || (cache_dtype != dtype && cache_dtype != PKV_E4M3)) return PKV_ERR_UNSUPPORTED;
    if (num_q_heads > (1 << 20) || rot_dim > head_dim || rot_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if (!q_weight != !k_weight) return PKV_ERR_ARG;
    if (q_weight && !(eps >= 0.f && std::isfinite(eps))) return PKV_ERR_ARG;
    const int vec = 16 / elem_bytes(dtype);
    if (q_stride < (int64_t)num_q_heads * head_dim || k_stride < (int64_t)num_kv_heads * head_dim ||
        v_stride < (int64_t)num_kv_heads * head_dim)
        return PKV_ERR_ARG;
    if (q_stride % vec != 0 || k_stride % vec != 0 || v_stride % vec != 0) return PKV_ERR_ALIGN;
    if (num_tokens == 0) return PKV_OK;
    if (!q_out || !q || !k || !v || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_ARG;
    if (rot_dim > 0 && (!positions || !inv_freq || num_axes <= 0)) return PKV_ERR_ARG;
    if (!aligned16(q_out) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned16(q_weight) || !aligned16(k_weight))
        return PKV_ERR_ALIGN;
    // rows may be turned in place only where each is read by the lanes that write it; what every token reads, and
    // what other warps write, may not lie under q_out at all
    const int eb = elem_bytes(dtype);
    auto bytes = [&](int64_t stride, int heads) {  // of a tensor's rows, the gaps between them included
        return (size_t)((num_tokens - 1) * stride + (int64_t)heads * head_dim) * eb;
    };
    const int64_t dense = (int64_t)num_q_heads * head_dim;
    const size_t out_bytes = bytes(dense, num_q_heads);
    if ((!(q_out == q && q_stride == dense) && overlaps(q_out, out_bytes, q, bytes(q_stride, num_q_heads))) ||
        overlaps(q_out, out_bytes, k, bytes(k_stride, num_kv_heads)) ||
        overlaps(q_out, out_bytes, v, bytes(v_stride, num_kv_heads)))
        return PKV_ERR_OVERLAP;
    const size_t weight_bytes = q_weight ? (size_t)head_dim * eb : 0, freq_bytes = (size_t)rot_dim / 2 * 4;
    const size_t cache_bytes = (size_t)num_blocks * num_kv_heads * tile_vecs(cache_dtype, head_dim) * 16;
    const struct {
        const void *p;
        size_t bytes;
    } others[] = {{q_weight, weight_bytes}, {k_weight, weight_bytes}, {slot_mapping, (size_t)num_tokens * 8},
                  {positions, freq_bytes > 0 ? (size_t)num_axes * num_tokens * 8 : 0}, {inv_freq, freq_bytes},
                  {axes, axes ? freq_bytes : 0}, {k_cache, cache_bytes}, {v_cache, cache_bytes}};
    for (const auto &o : others)
        if (o.bytes > 0 && overlaps(q_out, out_bytes, o.p, o.bytes)) return PKV_ERR_OVERLAP;
    pkv::RopeParams p{q_out, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, positions, inv_freq, axes,
                      slot_mapping, k_cache, v_cache, eps, num_axes, rot_dim, num_tokens, num_q_heads, num_kv_heads,
                      num_blocks, 1};
    const bool e4 = cache_dtype == PKV_E4M3, il = interleaved != 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == PKV_BF16)
        return head_dim == 128 ? launch_rope<__nv_bfloat16, 128>(p, il, e4, st)
                               : launch_rope<__nv_bfloat16, 64>(p, il, e4, st);
    return head_dim == 128 ? launch_rope<float, 128>(p, il, e4, st) : launch_rope<float, 64>(p, il, e4, st);
}

int tree_masks(int64_t *tree_mask, const int32_t *parents, const int32_t *query_start, int num_seqs, int num_queries,
               int max_query_len, void *stream) {
    if (num_seqs < 0 || num_queries < 0 || max_query_len < 0) return PKV_ERR_ARG;
    if (max_query_len > PKV_TREE_MAX_DRAFTS) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_queries == 0 || max_query_len == 0) return PKV_OK;
    if (!tree_mask || !parents || !query_start) return PKV_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(tree_mask) & 7) != 0) return PKV_ERR_ALIGN;
    const size_t mask_bytes = (size_t)num_queries * ((max_query_len + 63) / 64) * 8;
    if (overlaps(tree_mask, mask_bytes, parents, (size_t)num_queries * 4) ||
        overlaps(tree_mask, mask_bytes, query_start, ((size_t)num_seqs + 1) * 4))
        return PKV_ERR_OVERLAP;
    pkv::tree_masks_kernel<<<num_seqs, 64, 0, static_cast<cudaStream_t>(stream)>>>(
        tree_mask, parents, query_start, num_queries, max_query_len, (max_query_len + 63) / 64);
    return check_launch();
}

size_t pkv_tree_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_query_len,
                                int max_context_len) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || max_query_len <= 0 ||
        num_q_heads % num_kv_heads != 0 || tree_whole_units(max_context_len))
        return 0;
    const size_t rows = tree_pair(num_q_heads / num_kv_heads, max_query_len) ? 256 : 128;
    return kCounterBytes + kPersistMaxCtas * (sizeof(pkv::TreeCut) + 2 * rows * (2 + (size_t)head_dim) * sizeof(float));
}

int paged_tree_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                         const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start,
                         const int64_t *tree_mask, int mask_words, float scale, int num_kv_heads, int num_seqs,
                         int num_q_heads, int head_dim, int max_blocks_per_seq, int num_blocks, int num_queries,
                         int max_query_len, int max_context_len, pkv_dtype dtype, void *workspace,
                         size_t workspace_bytes, void *stream) {
    pkv::TreeParams tp{};
    int rc;
    if ((rc = attention_params(tp.d, out, q, k_cache, v_cache, block_tables, context_lens, scale, num_kv_heads,
                               num_seqs, num_q_heads, head_dim, max_blocks_per_seq, num_blocks, max_context_len,
                               64)) != PKV_OK)
        return rc;
    if (max_query_len < 0 || num_queries < 0 || mask_words < (max_query_len + 63) / 64) return PKV_ERR_ARG;
    if (dtype != PKV_BF16 || max_query_len > PKV_TREE_MAX_DRAFTS) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || max_query_len == 0 || num_queries == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !tree_mask)
        return PKV_ERR_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(tree_mask) & 7) != 0) return PKV_ERR_ALIGN;
    const size_t need = pkv_tree_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len,
                                                 max_context_len);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return PKV_ERR_WORKSPACE;
    tp.query_start = query_start;
    tp.mask = tree_mask;
    tp.mask_words = mask_words;
    tp.num_queries = num_queries;
    tp.max_query_len = max_query_len;
    const int g = tp.d.group, tile_tokens = 128 / g;
    alignas(64) CUtensorMap tmq, tmk, tmv;
    const int q_tokens = max_query_len < tile_tokens ? max_query_len : tile_tokens;  // loaded of a tile's drafts
    if ((rc = encode_q_map(&tmq, q, num_queries, num_q_heads, head_dim, g, q_tokens)) != PKV_OK) return rc;
    if ((rc = encode_cache_map(&tmk, k_cache, num_blocks, num_kv_heads, head_dim, true)) != PKV_OK) return rc;
    if ((rc = encode_cache_map(&tmv, v_cache, num_blocks, num_kv_heads, head_dim)) != PKV_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool pair = tree_pair(g, max_query_len);
    if (head_dim == 128)
        return pair ? launch_tree<128, true>(tmq, tmk, tmv, tp, q_tokens, workspace, st)
                    : launch_tree<128, false>(tmq, tmk, tmv, tp, q_tokens, workspace, st);
    return pair ? launch_tree<64, true>(tmq, tmk, tmv, tp, q_tokens, workspace, st)
                : launch_tree<64, false>(tmq, tmk, tmv, tp, q_tokens, workspace, st);
}

int kv_accept_layers(void *const *k_caches, void *const *v_caches, int num_layers, const int32_t *block_tables,
                     const int32_t *context_lens, const int32_t *query_start, const int32_t *accepted,
                     int max_accepted, const int32_t *num_accepted, int32_t *new_lens, int num_seqs,
                     int num_kv_heads, int head_dim, int max_blocks_per_seq, int num_blocks, pkv_dtype dtype,
                     void *stream) {
    if (num_layers < 0 || num_seqs < 0 || max_accepted < 0 || max_blocks_per_seq <= 0) return PKV_ERR_ARG;
    int rc;
    if ((rc = check_pool(num_kv_heads, num_blocks, head_dim)) != PKV_OK) return rc;
    if (!dtype_ok(dtype) || max_accepted > PKV_MAX_ACCEPTED || num_layers > 65535 || num_seqs > 65535 ||
        max_blocks_per_seq > INT32_MAX / 16)
        return PKV_ERR_UNSUPPORTED;
    if (num_layers == 0 || num_seqs == 0) return PKV_OK;
    if (!k_caches || !v_caches || !block_tables || !context_lens || !query_start || !num_accepted || !new_lens ||
        (max_accepted > 0 && !accepted))
        return PKV_ERR_ARG;
    const size_t lens = (size_t)num_seqs * 4;  // every CTA reads these after some have written
    if (overlaps(new_lens, lens, context_lens, lens) || overlaps(new_lens, lens, num_accepted, lens) ||
        overlaps(new_lens, lens, query_start, lens + 4) ||
        (max_accepted > 0 && overlaps(new_lens, lens, accepted, lens * max_accepted)) ||
        overlaps(new_lens, lens, block_tables, lens * max_blocks_per_seq))
        return PKV_ERR_OVERLAP;
    const int row_vecs = head_dim * elem_bytes(dtype) / 16;
    // heads of a CTA: as many as 12 KiB hold the rows of, one at least (64 accepted rows of 512 bytes take 64 KiB). More
    // heads share the lookups, fewer leave more CTAs: 64 sequences and 32 layers of 8 heads with 6 rows 13.6 us (17.8 with
    // 4 KiB, 15.4 with 48), with 16 rows 34.8 (34.9, 70); 8 sequences 5.7 (4.6, 8.1).
    const int head_bytes = 2 * max_accepted * row_vecs * 16;
    int heads = head_bytes > 0 ? 12288 / head_bytes : num_kv_heads;
    heads = heads < 1 ? 1 : heads > num_kv_heads ? num_kv_heads : heads;
    pkv::AcceptParams p{k_caches, v_caches, block_tables, context_lens, query_start, accepted, num_accepted, new_lens,
                        max_accepted, num_kv_heads, max_blocks_per_seq, num_blocks, row_vecs, heads};
    const size_t smem = (size_t)heads * head_bytes;  // at most 64 KiB
    static thread_local int configured_device = -1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    if (configured_device != dev) {
        if (cudaFuncSetAttribute(pkv::kv_accept_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 2 * PKV_MAX_ACCEPTED * 128 * 4) != cudaSuccess)
            return PKV_ERR_CUDA;
        configured_device = dev;
    }
    pkv::kv_accept_kernel<<<dim3((num_kv_heads + heads - 1) / heads, num_layers, num_seqs), 128, smem,
                            static_cast<cudaStream_t>(stream)>>>(p);
    return check_launch();
}

// The workspace of paged_decode_attention_common_prefix: the decode workspace of the persistent kernel, the tree kernel's
// records and states (its own counter header unused), the plan, and the rows' states of the prefix.
static size_t common_prefix_sums(int num_seqs, int num_q_heads) {  // (the outputs behind them are written 16 bytes at a time)
    return ((size_t)num_seqs * num_q_heads * 2 * sizeof(float) + 255) / 256 * 256;
}
static size_t common_prefix_plan_bytes(int num_seqs) { return (2 * (size_t)num_seqs * sizeof(int32_t) + 255) / 256 * 256; }
static size_t common_prefix_tree_bytes(int head_dim) {
    return kCounterBytes + kPersistMaxCtas * (sizeof(pkv::TreeCut) + 2 * 256 * (2 + (size_t)head_dim) * sizeof(float));
}

size_t pkv_common_prefix_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_q_heads % num_kv_heads != 0)
        return 0;
    return (persist_workspace_bytes(num_q_heads, num_kv_heads, head_dim) + 255) / 256 * 256 +
           common_prefix_tree_bytes(head_dim) + common_prefix_plan_bytes(num_seqs) +
           common_prefix_sums(num_seqs, num_q_heads) + (size_t)num_seqs * num_q_heads * head_dim * sizeof(float);
}

int paged_decode_attention_common_prefix(void *out, const void *q, const void *k_cache, const void *v_cache,
                                         const int32_t *block_tables, const int32_t *context_lens, float scale,
                                         int num_kv_heads, int num_seqs, int num_q_heads, int head_dim,
                                         int max_blocks_per_seq, int num_blocks, int max_context_len,
                                         const int32_t *group_start, const int32_t *shared_blocks, int num_groups,
                                         int max_group_size, pkv_dtype dtype, void *workspace, size_t workspace_bytes,
                                         void *stream) {
    pkv::DecodeParams p{};
    int rc;
    if ((rc = attention_params(p, out, q, k_cache, v_cache, block_tables, context_lens, scale, num_kv_heads, num_seqs,
                               num_q_heads, head_dim, max_blocks_per_seq, num_blocks, max_context_len, 16)) != PKV_OK)
        return rc;
    if (num_groups < 0 || max_group_size < 0 || num_groups > num_seqs) return PKV_ERR_ARG;
    if (dtype != PKV_BF16 || num_seqs > kPersistMaxSeqs) return PKV_ERR_UNSUPPORTED;
    // the decode kernel counts a launch's blocks in 32 bits
    if (std::min<int64_t>(((int64_t)max_context_len + 15) / 16, max_blocks_per_seq) * num_seqs > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PKV_ERR_ARG;
    if (num_groups > 0 && (!group_start || !shared_blocks)) return PKV_ERR_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ALIGN;
    const size_t need = pkv_common_prefix_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return PKV_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    p.counters = reinterpret_cast<int *>(ws);
    p.partials = reinterpret_cast<float *>(ws + kCounterBytes);
    ws += (persist_workspace_bytes(num_q_heads, num_kv_heads, head_dim) + 255) / 256 * 256;
    char *tree = ws;
    ws += common_prefix_tree_bytes(head_dim);
    int32_t *tokens = reinterpret_cast<int32_t *>(ws), *first_blocks = tokens + num_seqs;
    ws += common_prefix_plan_bytes(num_seqs);
    float *prefix_ml = reinterpret_cast<float *>(ws);
    float *prefix_o = reinterpret_cast<float *>(ws + common_prefix_sums(num_seqs, num_q_heads));
    p.first_blocks = first_blocks;
    p.prefix_ml = prefix_ml;
    p.prefix_o = prefix_o;

    const int g = p.group, tile_tokens = 128 / g;
    alignas(64) CUtensorMap tmq, tmk, tmk_half, tmv;
    if ((rc = encode_cache_map(&tmk, k_cache, num_blocks, num_kv_heads, head_dim)) != PKV_OK) return rc;
    if ((rc = encode_cache_map(&tmv, v_cache, num_blocks, num_kv_heads, head_dim)) != PKV_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    pkv::common_prefix_plan_kernel<<<1, 1024, 0, st>>>(p, group_start, shared_blocks, num_groups, max_group_size, tokens,
                                                       first_blocks);
    if ((rc = check_launch()) != PKV_OK) return rc;
    if (num_groups > 0 && max_group_size > 0) {
        const int q_tokens = max_group_size < tile_tokens ? max_group_size : tile_tokens;
        if ((rc = encode_q_map(&tmq, q, num_seqs, num_q_heads, head_dim, g, q_tokens)) != PKV_OK) return rc;
        if ((rc = encode_cache_map(&tmk_half, k_cache, num_blocks, num_kv_heads, head_dim, true)) != PKV_OK) return rc;
        pkv::TreeParams tp{};
        tp.d = p;
        tp.d.context_lens = tokens;
        tp.d.num_seqs = num_groups;
        tp.query_start = group_start;
        tp.num_queries = num_seqs;
        tp.max_query_len = max_group_size;
        tp.prefix_ml = prefix_ml;
        tp.prefix_o = prefix_o;
        const bool pair = tree_pair(g, max_group_size);
        rc = head_dim == 128 ? (pair ? launch_tree<128, true, true>(tmq, tmk_half, tmv, tp, q_tokens, tree, st)
                                     : launch_tree<128, false, true>(tmq, tmk_half, tmv, tp, q_tokens, tree, st))
                             : (pair ? launch_tree<64, true, true>(tmq, tmk_half, tmv, tp, q_tokens, tree, st)
                                     : launch_tree<64, false, true>(tmq, tmk_half, tmv, tp, q_tokens, tree, st));
        if (rc != PKV_OK) return rc;
    }
    constexpr int ns128 = PKV_PERSIST_STAGES_D128, ns64 = PKV_PERSIST_STAGES_D64;
    return persistent_by_shape<__nv_bfloat16, ns128, ns64, kPersistWarps, pkv::kBehindPrefix>(
        tmk, tmv, p, st, num_groups > 0 && max_group_size > 0, head_dim, g);
}

int paged_decode_attention_scored(void *out, const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *block_tables, const int32_t *context_lens, float scale, float softcap,
                                  int window, const float *slopes, int num_kv_heads, int num_seqs, int num_q_heads,
                                  int head_dim, int max_blocks_per_seq, int num_blocks, int max_context_len,
                                  pkv_dtype dtype, int partition_tokens, void *workspace, size_t workspace_bytes,
                                  void *stream) {
    const ScoreArgs scores{softcap, window, slopes};
    return decode_dispatch(out, q, k_cache, v_cache, block_tables, context_lens, scale, num_kv_heads, num_seqs,
                           num_q_heads, head_dim, max_blocks_per_seq, num_blocks, max_context_len, dtype,
                           partition_tokens, workspace, workspace_bytes, stream, kLaunch, &scores);
}

int paged_prefill_attention_scored(void *out, const void *q, const void *k_cache, const void *v_cache,
                                   const int32_t *block_tables, const int32_t *context_lens,
                                   const int32_t *query_start, float scale, float softcap, int window,
                                   const float *slopes, const int32_t *prefix_lens, int num_kv_heads, int num_seqs,
                                   int num_q_heads, int head_dim, int max_blocks_per_seq, int num_blocks,
                                   int num_queries, int max_query_len, int max_context_len, pkv_dtype dtype,
                                   void *stream) {
    pkv::ScoredPrefillParams sp{};
    pkv::PrefillParams &pp = sp.pp;
    int rc;
    if ((rc = attention_params(pp.d, out, q, k_cache, v_cache, block_tables, context_lens, scale, num_kv_heads,
                               num_seqs, num_q_heads, head_dim, max_blocks_per_seq, num_blocks, max_context_len,
                               64)) != PKV_OK)
        return rc;
    if (max_query_len < 0 || num_queries < 0) return PKV_ERR_ARG;
    if ((rc = score_params(pp.d, {softcap, window, slopes}, scale)) != PKV_OK) return rc;
    if (dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(prefix_lens) & 3) != 0) return PKV_ERR_ALIGN;
    const int g = pp.d.group, tile_tokens = 128 / g;
    const long long pairs = (max_query_len + 2LL * tile_tokens - 1) / (2 * tile_tokens);
    if (pairs > 65535) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || max_query_len == 0 || num_queries == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start) return PKV_ERR_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ALIGN;
    if (window == 0) pp.d.window = INT32_MAX;
    sp.near_max = pkv::capped_near_max(pp.d.scale_log2, pp.d.cap_in);
    sp.prefix_lens = prefix_lens;
    pp.query_start = query_start;
    pp.tile_tokens = tile_tokens;
    pp.max_query_len = max_query_len;
    pp.num_queries = num_queries;
    // CTA order as for paged_prefill_attention
    pp.seq_major = max_context_len >= 2LL * max_query_len ? 1 : 0;
    const dim3 grid = pp.seq_major ? dim3(num_kv_heads, (unsigned)pairs, num_seqs)
                                   : dim3(num_kv_heads, num_seqs, (unsigned)pairs);
    alignas(64) CUtensorMap tmq, tmk, tmv;
    if ((rc = encode_q_map(&tmq, q, num_queries, num_q_heads, head_dim, g, tile_tokens)) != PKV_OK) return rc;
    if ((rc = encode_cache_map(&tmk, k_cache, num_blocks, num_kv_heads, head_dim, true)) != PKV_OK) return rc;
    if ((rc = encode_cache_map(&tmv, v_cache, num_blocks, num_kv_heads, head_dim)) != PKV_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // At most so many pairs hold tokens. A pair sees its tokens and what the window leaves before them and, under
    // prefixes, behind.
    const long long in_use = num_kv_heads * std::min(pairs * num_seqs, num_queries / (2LL * tile_tokens) + num_seqs);
    const long long seen = std::min<long long>(max_context_len, 2LL * tile_tokens + (prefix_lens ? 2LL : 1LL) * pp.d.window);
    return head_dim == 128 ? launch_prefill_scored<128>(tmq, tmk, tmv, sp, grid, in_use, seen / 128 + 1, st)
                           : launch_prefill_scored<64>(tmq, tmk, tmv, sp, grid, in_use, seen / 128 + 1, st);
}

int verify_drafts(int32_t *accepted, int max_accepted, int32_t *num_accepted, int64_t *next_tokens,
                  const int64_t *tokens, const int32_t *parents, const int32_t *query_start, const void *target_probs,
                  int64_t target_stride, const void *draft_probs, int64_t draft_stride, const float *uniforms,
                  const float *final_uniforms, int num_seqs, int num_queries, int max_query_len, int vocab,
                  pkv_dtype dtype, void *stream) {
    if (num_seqs < 0 || num_queries < 0 || max_query_len < 0 || max_accepted < 1 || vocab <= 0) return PKV_ERR_ARG;
    if (!dtype_ok(dtype) || max_query_len > PKV_TREE_MAX_DRAFTS || vocab > (1 << 30) || num_seqs > (1 << 24))
        return PKV_ERR_UNSUPPORTED;
    if (target_stride < vocab || (draft_probs && draft_stride < vocab)) return PKV_ERR_ARG;
    const int eb = elem_bytes(dtype);
    const int64_t most = (INT64_MAX / 8) / (num_queries > 0 ? num_queries : 1);  // (rows' bytes fit 63 bits)
    if (target_stride > most || (draft_probs && draft_stride > most)) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!accepted || !num_accepted || !next_tokens || !query_start || !final_uniforms) return PKV_ERR_ARG;
    if (num_queries > 0 && (!tokens || !parents || !target_probs || !uniforms)) return PKV_ERR_ARG;
    auto off = [](const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; };
    if (off(accepted, 4) || off(num_accepted, 4) || off(next_tokens, 8) || off(tokens, 8) || off(parents, 4) ||
        off(query_start, 4) || off(target_probs, eb) || off(draft_probs, eb) || off(uniforms, 4) ||
        off(final_uniforms, 4))
        return PKV_ERR_ALIGN;
    auto row_bytes = [&](int64_t stride) { return num_queries > 0 ? (size_t)((num_queries - 1) * stride + vocab) * eb : 0; };
    const size_t seqs = num_seqs, rows = num_queries;
    const struct {
        const void *p;
        size_t bytes;
    } all[] = {{accepted, seqs * max_accepted * 4}, {num_accepted, seqs * 4}, {next_tokens, seqs * 8},
               {tokens, rows * 8}, {parents, rows * 4}, {query_start, (seqs + 1) * 4},
               {target_probs, row_bytes(target_stride)}, {draft_probs, draft_probs ? row_bytes(draft_stride) : 0},
               {uniforms, rows * 4}, {final_uniforms, seqs * 4}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < (int)(sizeof(all) / sizeof(all[0])); ++j)
            if (all[j].bytes > 0 && overlaps(all[i].p, all[i].bytes, all[j].p, all[j].bytes)) return PKV_ERR_OVERLAP;
    const bool vector_rows = aligned16(target_probs) && target_stride * eb % 16 == 0 &&
                             (!draft_probs || (aligned16(draft_probs) && draft_stride * eb % 16 == 0));
    const pkv::VerifyParams p{accepted, num_accepted, next_tokens, tokens, parents, query_start, target_probs, draft_probs,
                              target_stride, draft_stride, uniforms, final_uniforms, num_queries, max_query_len,
                              max_accepted, vocab, vector_rows ? 1 : 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PKV_BF16 ? launch_verify<__nv_bfloat16>(p, num_seqs, st) : launch_verify<float>(p, num_seqs, st);
}

}  // extern "C"
