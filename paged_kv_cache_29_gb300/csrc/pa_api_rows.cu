// pa_api_rows.cu -- the C ABI of the calls that say which rows of a cache count
// (pa_decode_sinks, pa_decode_weights, pa_evict, pa_verify_draft): argument checks,
// workspace layouts and launches. Everything here runs on the host and only enqueues
// work on the caller's stream.
#include <climits>
#include <cmath>
#include <cstdint>

#include "pa_internal.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Heads of a token that these calls take, and query columns (heads per KV head x query
// tokens): products of them with rows and dims stay below 2^31.
constexpr int kMaxHeads = 1 << 20;
constexpr int kMaxColumns = 1024;
// Row numbers stay below 2^31 with a partition's rows added.
constexpr int kMaxRows = INT_MAX - 4096;
constexpr int kMaxVocab = 1 << 22;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
cudaStream_t stream_of(struct CUstream_st* s) { return reinterpret_cast<cudaStream_t>(s); }

// Workspace of one launch of at most kPlanMaxSeqs sequences, as pa_decode lays it
// out: 256 bytes (the number of work items first), the work items, the partitions' maxima and sums, their outputs;
// pa_decode_weights has the maxima and sums of single partitions too, those of whole
// sequences, and the scores.
struct Layout {
    size_t items, ml, o, final_ml, scores, total;
};

Layout layout_for(long long num_seqs, long long num_heads, int head_dim, int max_context_len, long long parts,
                  int num_queries, bool weights) {
    const long long seqs = num_seqs < pa::kPlanMaxSeqs ? num_seqs : pa::kPlanMaxSeqs;
    const size_t units = static_cast<size_t>(seqs) * num_heads * parts;
    const size_t prows = units * static_cast<size_t>(num_queries);
    Layout w;
    w.items = 256;
    w.ml = w.items + 16 * units;
    w.o = w.ml + (weights || parts > 1 ? 8 * prows : 0);
    w.final_ml = w.o + (parts > 1 ? 4 * prows * static_cast<size_t>(head_dim) : 0);
    if (weights) w.final_ml = (w.final_ml + 15) / 16 * 16;
    w.scores = w.final_ml + (weights ? (8 * static_cast<size_t>(seqs) * num_heads * num_queries + 15) / 16 * 16 : 0);
    w.total = w.scores + (weights ? 4 * static_cast<size_t>(seqs) * num_heads * num_queries *
                                        ((static_cast<size_t>(max_context_len) + 15) / 16 * 16)
                                  : 0);
    return w;
}

// pa_decode_sinks (row_weights null) and pa_decode_weights (window 0).
pa_status rows_call(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                    const int32_t* context_lens, float scale, int window, int num_sinks, void* out,
                    float* row_weights, int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                    int head_dim, int block_size, int num_blocks, int max_blocks_per_seq,
                    int max_context_len, pa_dtype dtype, void* workspace, size_t workspace_bytes,
                    int32_t* error_word, bool weights, struct CUstream_st* stream, int withhold_tile = -1) {
    if (num_seqs < 0 || num_queries < 1 || num_queries > 8 || num_heads <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq < 0 ||
        max_context_len < 0 || num_heads % num_kv_heads != 0 || !std::isfinite(scale) ||
        (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16))
        return PA_ERR_INVALID_ARG;
    if (static_cast<long long>(max_context_len) > static_cast<long long>(max_blocks_per_seq) * block_size)
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (head_dim > pa::kMaxHeadDim || num_heads > kMaxHeads ||
        static_cast<long long>(group) * num_queries > kMaxColumns || max_context_len > kMaxRows)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out || (weights && !row_weights) ||
        !aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(row_weights, 4))
        return PA_ERR_INVALID_ARG;
    // The rows that any of the Q tokens' windows holds. A window that no row can be
    // outside of is none.
    const bool all = weights || window >= max_context_len;
    const int rows_seen = all ? 0 : window + num_queries - 1;
    const int sinks = all ? 0 : (num_sinks < max_context_len ? num_sinks : max_context_len);
    // Rows of the longest sequence's partitions: its first rows in whole tiles,
    // its windows' and up to 15 before them in the same tile.
    const long long seen = (static_cast<long long>(window) + num_queries + 29) / 16 * 16 + (static_cast<long long>(num_sinks) + 15) / 16 * 16;
    const long long most = all || seen > max_context_len ? max_context_len : seen;
    // A window's rows in equal partitions of 512 rows or more: 128 sequences with a window
    // of 1,024 rows and 4 first ones, 1,056 with their tiles, take 87 us in two partitions, 91
    // in 512 + 512 + 32. By the window and the first rows alone, so that a sequence's partitions do
    // not depend on the batch, nor on the bound on its lengths.
    int P = pa::kDefaultPartition;                // (752 at most)
    if (!weights) {
        const long long equal = (seen + P / 2) / P;
        const long long rows = equal > 0 ? ceil_div(ceil_div(seen, equal), 16) * 16 : 0;
        if (rows > P) P = static_cast<int>(rows);
    }
    const long long parts = most > 0 ? ceil_div(most, P) : 1;
    const long long chunk = num_seqs < pa::kPlanMaxSeqs ? num_seqs : pa::kPlanMaxSeqs;
    if (parts * chunk * num_kv_heads > 0x3fffffffLL) return PA_ERR_UNSUPPORTED;
    const Layout lay = layout_for(num_seqs, num_heads, head_dim, max_context_len, parts, num_queries, weights);
    const size_t asked = weights ? lay.total
                                 : pa_decode_workspace_size_multi(num_seqs, num_queries, num_heads,
                                                                  head_dim, max_context_len);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < asked) return PA_ERR_WORKSPACE;

    uint8_t* ws = static_cast<uint8_t*>(workspace);
    pa::DecodeParams base{};
    base.k_cache = k_cache;
    base.v_cache = v_cache;
    base.items = reinterpret_cast<int4*>(ws + lay.items);
    if (weights || parts > 1) base.part_ml = reinterpret_cast<float*>(ws + lay.ml);
    if (parts > 1) base.part_o = reinterpret_cast<float*>(ws + lay.o);
    if (weights) {
        base.row_weights = row_weights;
        base.final_ml = reinterpret_cast<float2*>(ws + lay.final_ml);
        base.scores = reinterpret_cast<float*>(ws + lay.scores);
        base.score_rows = (max_context_len + 15) / 16 * 16;
        base.item_count = reinterpret_cast<int32_t*>(ws);
    }
    base.error_word = error_word;
    base.withhold_tile = withhold_tile;
    base.scale_log2 = scale * kLog2e;
    base.k_scale = base.v_scale = 1.0f;
    base.num_queries = num_queries;
    base.window = rows_seen;
    base.num_sinks = sinks;
    base.num_heads = num_heads;
    base.num_kv_heads = num_kv_heads;
    base.head_dim = head_dim;
    base.block_size = block_size;
    base.num_blocks = num_blocks;
    base.max_blocks_per_seq = max_blocks_per_seq;
    base.context_cap = max_context_len;
    base.partition_size = base.partition_long = P;
    base.partition_long_from = pa::kNoLongPartitions;
    base.max_parts = static_cast<int>(parts);
    const size_t es = dtype == PA_DTYPE_F32 ? 4 : 2;
    const long long pool_rows = static_cast<long long>(num_blocks) * num_kv_heads * block_size;
    // The tile ring, where an item takes whole heads of at least one token, and the items of
    // all column groups fit the work list (sized for one per query head).
    const int tokens = pa::rows_group_tokens(dtype, head_dim, group, num_queries);
    const int groups = tokens > 0 ? static_cast<int>(ceil_div(num_queries, tokens)) : 0;
    const bool ring = block_size % 16 == 0 && pool_rows < INT_MAX && groups > 0 && groups <= group &&
                      parts * chunk * num_kv_heads * groups <= 0x3fffffffLL;
    base.col_groups = groups;
    base.group_tokens = tokens;
    CUtensorMap tk, tv;
    int sms = 0;
    if (ring) {
        pa_status ps = pa::make_pool_map(&tk, k_cache, dtype, head_dim, pool_rows);
        if (ps == PA_OK) ps = pa::make_pool_map(&tv, v_cache, dtype, head_dim, pool_rows);
        if (ps != PA_OK) return ps;
        sms = pa::device_sms();
        if (sms <= 0) return PA_ERR_CUDA;
    }
    // Batches above kPlanMaxSeqs sequences run as consecutive launches over
    // slices of the batch; they reuse the workspace in stream order.
    for (int s0 = 0; s0 < num_seqs; s0 += pa::kPlanMaxSeqs) {
        pa::DecodeParams p = base;
        const size_t qoff = static_cast<size_t>(s0) * num_queries * num_heads * head_dim * es;
        p.q = static_cast<const uint8_t*>(q) + qoff;
        p.out = static_cast<uint8_t*>(out) + qoff;
        p.block_tables = block_tables + static_cast<size_t>(s0) * max_blocks_per_seq;
        p.context_lens = context_lens + s0;
        p.num_seqs = num_seqs - s0 < pa::kPlanMaxSeqs ? num_seqs - s0 : pa::kPlanMaxSeqs;
        // With one partition each, and each row's columns in one item, the tile ring adds the row
        // weights too, while its CTAs (up to four an SM) take two items each or about that: in
        // more items their tiles wait for it (up to 512 rows and 8 KV heads: 9.6 us instead of
        // 11.5 for one sequence, 53 instead of 57 for 128, but 100 as without for 250 and 214 instead of 204
        // for 600).
        const bool ends = weights && ring && parts == 1 && groups == 1 && 1LL * p.num_seqs * num_kv_heads <= 8LL * sms;
        const cudaError_t err = !ring     ? pa::launch_decode_rows(p, dtype, stream_of(stream))
                                : ends    ? pa::launch_decode_weights_short(tk, tv, p, dtype, sms, stream_of(stream))
                                : weights ? pa::launch_decode_weights(tk, tv, p, dtype, sms, stream_of(stream))
                                          : pa::launch_decode_sinks(tk, tv, p, dtype, sms, stream_of(stream));
        if (err != cudaSuccess) return PA_ERR_CUDA;
        if (parts > 1 && pa::launch_combine(p, dtype, stream_of(stream), true) != cudaSuccess) return PA_ERR_CUDA;
        if (weights && !ends && pa::launch_row_weights(p, ring ? p.item_count : nullptr, stream_of(stream)) != cudaSuccess)
            return PA_ERR_CUDA;
    }
    return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_decode_sinks(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens, float scale,
                          int window, int num_sinks, void* out, int num_seqs, int num_queries,
                          int num_heads, int num_kv_heads, int head_dim, int block_size,
                          int num_blocks, int max_blocks_per_seq, int max_context_len,
                          pa_dtype dtype, void* workspace, size_t workspace_bytes,
                          int32_t* error_word, struct CUstream_st* stream) {
    if (window < 1 || num_sinks < 0) return PA_ERR_INVALID_ARG;
    return rows_call(q, k_cache, v_cache, block_tables, context_lens, scale, window, num_sinks, out, nullptr,
                     num_seqs, num_queries, num_heads, num_kv_heads, head_dim, block_size, num_blocks,
                     max_blocks_per_seq, max_context_len, dtype, workspace, workspace_bytes, error_word,
                     false, stream);
}

pa_status pa_decode_weights(const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens, float scale,
                            void* out, float* row_weights, int num_seqs, int num_queries,
                            int num_heads, int num_kv_heads, int head_dim, int block_size,
                            int num_blocks, int max_blocks_per_seq, int max_context_len,
                            pa_dtype dtype, void* workspace, size_t workspace_bytes,
                            int32_t* error_word, struct CUstream_st* stream) {
    return rows_call(q, k_cache, v_cache, block_tables, context_lens, scale, 0, 0, out, row_weights, num_seqs,
                     num_queries, num_heads, num_kv_heads, head_dim, block_size, num_blocks,
                     max_blocks_per_seq, max_context_len, dtype, workspace, workspace_bytes, error_word,
                     true, stream);
}

pa_status pa_test_withhold_tile_weights(const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_tables, const int32_t* context_lens, float scale,
                                        void* out, float* row_weights, int num_seqs, int num_queries,
                                        int num_heads, int num_kv_heads, int head_dim, int block_size,
                                        int num_blocks, int max_blocks_per_seq, int max_context_len,
                                        pa_dtype dtype, void* workspace, size_t workspace_bytes,
                                        int32_t* error_word, int withhold_tile, struct CUstream_st* stream) {
    if (withhold_tile < 0 || error_word == nullptr) return PA_ERR_INVALID_ARG;
    return rows_call(q, k_cache, v_cache, block_tables, context_lens, scale, 0, 0, out, row_weights, num_seqs,
                     num_queries, num_heads, num_kv_heads, head_dim, block_size, num_blocks,
                     max_blocks_per_seq, max_context_len, dtype, workspace, workspace_bytes, error_word,
                     true, stream, withhold_tile);
}

size_t pa_decode_workspace_size_weights(int num_seqs, int num_queries, int num_heads, int head_dim,
                                        int max_context_len) {
    if (num_seqs <= 0 || num_queries <= 0 || num_heads <= 0 || head_dim <= 0 || max_context_len < 0) return 0;
    const long long parts = max_context_len > 0 ? ceil_div(max_context_len, pa::kDefaultPartition) : 1;
    return layout_for(num_seqs, num_heads, head_dim, max_context_len, parts, num_queries, true).total;
}

size_t pa_evict_workspace_size(int num_seqs, int num_kv_heads, int max_context_len) {
    if (num_seqs <= 0 || num_kv_heads <= 0 || max_context_len < 0) return 0;
    const size_t heads = static_cast<size_t>(num_seqs) * num_kv_heads;
    // the moves, then where they start per sequence and KV head, a length and a place per sequence
    return heads * max_context_len * sizeof(uint2) + 4 * (heads + 2 * static_cast<size_t>(num_seqs));
}

pa_status pa_evict(void* k_cache, void* v_cache, void* k_params, void* v_params, float* row_weights,
                   const int32_t* block_tables, const int32_t* context_lens, const int32_t* keep_lens,
                   const int32_t* out_tables, int32_t* lens_out, int num_sinks, int num_recent,
                   int num_seqs, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                   int max_blocks_per_seq, int max_context_len, pa_dtype dtype, void* workspace,
                   size_t workspace_bytes, int32_t* error_word, struct CUstream_st* stream) {
    if (num_sinks < 0 || num_recent < 0 || num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq < 0 || max_context_len < 0 ||
        dtype < PA_DTYPE_F32 || dtype > PA_DTYPE_INT4)
        return PA_ERR_INVALID_ARG;
    if (static_cast<long long>(max_context_len) > static_cast<long long>(max_blocks_per_seq) * block_size)
        return PA_ERR_INVALID_ARG;
    const long long row_bytes = dtype == PA_DTYPE_F32    ? 4LL * head_dim
                                : dtype == PA_DTYPE_BF16 ? 2LL * head_dim
                                : dtype == PA_DTYPE_INT4 ? head_dim / 2
                                                         : head_dim;
    if ((dtype == PA_DTYPE_INT4 && head_dim % 2 != 0) || row_bytes % 16 != 0 || row_bytes > 4 * pa::kMaxHeadDim ||
        num_kv_heads > kMaxHeads || max_context_len > kMaxRows ||
        static_cast<double>(num_blocks) * num_kv_heads * block_size >= 4294967296.0 ||
        static_cast<long long>(num_seqs) * num_kv_heads > 0x3fffffLL)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    const bool params = dtype == PA_DTYPE_INT8 || dtype == PA_DTYPE_INT4;
    if (!k_cache || !v_cache || !row_weights || !block_tables || !context_lens || !keep_lens || !out_tables ||
        !lens_out || (params ? !k_params || !v_params : k_params || v_params))
        return PA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_params, 4) || !aligned(v_params, 4) ||
        !aligned(row_weights, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(keep_lens, 4) || !aligned(out_tables, 4) || !aligned(lens_out, 4))
        return PA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < pa_evict_workspace_size(num_seqs, num_kv_heads, max_context_len))
        return PA_ERR_WORKSPACE;
    const size_t heads = static_cast<size_t>(num_seqs) * num_kv_heads;
    pa::EvictParams p{};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_params = static_cast<uint32_t*>(k_params);
    p.v_params = static_cast<uint32_t*>(v_params);
    p.row_weights = row_weights;
    p.block_tables = block_tables;
    p.out_tables = out_tables;
    p.context_lens = context_lens;
    p.keep_lens = keep_lens;
    p.lens_out = lens_out;
    p.moves = static_cast<uint2*>(workspace);
    p.starts = reinterpret_cast<int32_t*>(p.moves + heads * max_context_len);
    p.new_lens = p.starts + heads;
    p.order = p.new_lens + num_seqs;
    p.error_word = error_word;
    p.num_sinks = num_sinks;
    p.num_recent = num_recent;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.row_bytes = static_cast<int>(row_bytes);
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_cap = max_context_len;
    p.by_block = pa::Divisor(static_cast<uint32_t>(block_size));
    return pa::launch_evict(p, stream_of(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_verify_draft(const float* target_probs, int64_t target_seq_stride, int64_t target_row_stride,
                          const float* draft_probs, int64_t draft_seq_stride, int64_t draft_row_stride,
                          const int32_t* draft_tokens, const int32_t* num_drafts, const float* uniforms,
                          int32_t* out_tokens, int32_t* num_accepted, const int32_t* context_lens,
                          int32_t* lens_out, int num_seqs, int max_drafts, int vocab_size,
                          int32_t* error_word, struct CUstream_st* stream) {
    if (num_seqs < 0 || max_drafts < 0 || vocab_size <= 0 || (context_lens == nullptr) != (lens_out == nullptr))
        return PA_ERR_INVALID_ARG;
    if (max_drafts > 64 || vocab_size > kMaxVocab || num_seqs > (1 << 24)) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!target_probs || !uniforms || !out_tokens || !num_accepted || (max_drafts > 0 && !draft_tokens))
        return PA_ERR_INVALID_ARG;
    if (!aligned(target_probs, 4) || !aligned(draft_probs, 4) || !aligned(draft_tokens, 4) ||
        !aligned(num_drafts, 4) || !aligned(uniforms, 4) || !aligned(out_tokens, 4) ||
        !aligned(num_accepted, 4) || !aligned(context_lens, 4) || !aligned(lens_out, 4))
        return PA_ERR_INVALID_ARG;
    pa::VerifyParams p{};
    p.target = target_probs;
    p.draft = draft_probs;
    p.target_seq = target_seq_stride;
    p.target_row = target_row_stride;
    p.draft_seq = draft_seq_stride;
    p.draft_row = draft_row_stride;
    p.tokens = draft_tokens;
    p.num_drafts = num_drafts;
    p.uniforms = uniforms;
    p.out_tokens = out_tokens;
    p.num_accepted = num_accepted;
    p.context_lens = context_lens;
    p.lens_out = lens_out;
    p.error_word = error_word;
    p.num_seqs = num_seqs;
    p.max_drafts = max_drafts;
    p.vocab = vocab_size;
    return pa::launch_verify(p, stream_of(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
