// pa_api_int4.cu -- the C ABI of the 4-bit cache calls and of the norm and
// rotation calls: argument checks and launches. Everything here runs on the
// host and only enqueues work on the caller's stream.
#include <climits>
#include <cmath>
#include <cstdint>

#include "pa_internal.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Heads of a token that these calls take: products of heads, lanes per row, query
// tokens and dims stay below 2^31 in the launches and kernels.
constexpr int kMaxHeads = 1 << 20;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
bool plain_dtype(int d) { return d == PA_DTYPE_F32 || d == PA_DTYPE_BF16; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

cudaStream_t stream_of(struct CUstream_st* s) { return reinterpret_cast<cudaStream_t>(s); }
pa_status status_of(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

// The pool of a 4-bit cache: present and aligned.
bool pool4_ok(const void* kc, const void* vc, const void* kp, const void* vp) {
    return kc && vc && kp && vp && aligned16(kc) && aligned16(vc) && aligned16(kp) && aligned16(vp);
}

// What the three norm and rotation calls share. PA_OK with p filled in, or
// the error; an empty call (num_tokens 0) is PA_OK too.
pa_status norm_rope_params(const pa_norm_rope_args* a, pa::NormRopeParams* p) {
    if (a == nullptr) return PA_ERR_INVALID_ARG;
    if (a->num_tokens < 0 || a->num_heads <= 0 || a->num_kv_heads <= 0 || a->head_dim <= 0 ||
        !plain_dtype(a->dtype) || !plain_dtype(a->weight_dtype) || !(a->eps >= 0.0f) ||
        a->eps == INFINITY || !std::isfinite(a->weight_offset) || a->rot_dim < 0 ||
        a->rot_dim > a->head_dim)
        return PA_ERR_INVALID_ARG;
    if (a->head_dim % 16 != 0 || a->head_dim > pa::kMaxHeadDim || a->rot_dim % 16 != 0 ||
        a->num_heads > kMaxHeads || a->num_kv_heads > kMaxHeads)
        return PA_ERR_UNSUPPORTED;
    if (a->rot_dim > 0) {
        if (a->num_axes < 1 || a->num_axes > 4 || a->max_position <= 0) return PA_ERR_INVALID_ARG;
        if (a->pair_axis != nullptr)
            for (int i = 0; i < a->rot_dim / 2; ++i)
                if (a->pair_axis[i] >= a->num_axes) return PA_ERR_INVALID_ARG;
    }
    if (a->num_tokens == 0) return PA_OK;
    const int64_t unit = 16 / (a->dtype == PA_DTYPE_F32 ? 4 : 2);   // elements in 16 bytes
    const int64_t q_row = static_cast<int64_t>(a->num_heads) * a->head_dim;
    const int64_t k_row = static_cast<int64_t>(a->num_kv_heads) * a->head_dim;
    if (!a->q || !a->k || !a->q_out || !aligned16(a->q) || !aligned16(a->k) ||
        !aligned16(a->q_out) || !aligned16(a->q_weight) || !aligned16(a->k_weight) ||
        a->q_stride < q_row || a->k_stride < k_row || a->q_out_stride < q_row ||
        a->q_stride % unit != 0 || a->k_stride % unit != 0 || a->q_out_stride % unit != 0)
        return PA_ERR_INVALID_ARG;
    if (a->rot_dim > 0 && (!a->cos_sin || !a->positions || !aligned16(a->cos_sin) || !aligned(a->positions, 4)))
        return PA_ERR_INVALID_ARG;
    p->q = a->q;
    p->k = a->k;
    p->q_stride = a->q_stride;
    p->k_stride = a->k_stride;
    p->q_out = a->q_out;
    p->q_out_stride = a->q_out_stride;
    p->q_weight = a->q_weight;
    p->k_weight = a->k_weight;
    p->weight_bf16 = a->weight_dtype == PA_DTYPE_BF16;
    p->eps = a->eps;
    p->weight_offset = a->weight_offset;
    p->cos_sin = a->cos_sin;
    p->positions = a->positions;
    p->num_tokens = a->num_tokens;
    p->num_heads = a->num_heads;
    p->num_kv_heads = a->num_kv_heads;
    p->head_dim = a->head_dim;
    p->rot_dim = a->rot_dim;
    p->max_position = a->max_position;
    p->num_axes = a->num_axes;
    p->interleaved = a->interleaved != 0;
    for (int i = 0; i < a->rot_dim / 2; ++i) p->pair_axis[i] = a->pair_axis ? a->pair_axis[i] : 0;
    return PA_OK;
}

// V rows and slots of the appending calls.
pa_status append_params(const pa_norm_rope_args* a, const void* v, int64_t v_stride,
                        const int64_t* slot_mapping, int block_size, int num_blocks,
                        int32_t* error_word, pa::NormRopeParams* p) {
    const int64_t unit = 16 / (a->dtype == PA_DTYPE_F32 ? 4 : 2);
    if (!v || !slot_mapping || !aligned16(v) || !aligned(slot_mapping, 8) ||
        v_stride < static_cast<int64_t>(a->num_kv_heads) * a->head_dim || v_stride % unit != 0)
        return PA_ERR_INVALID_ARG;
    p->v = v;
    p->v_stride = v_stride;
    p->slot_mapping = slot_mapping;
    p->block_size = block_size;
    p->num_slots = static_cast<long long>(num_blocks) * block_size;
    p->error_word = error_word;
    return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_reshape_and_cache_int4(const void* k_new, const void* v_new, pa_dtype new_dtype,
                                    const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                    void* k_params, void* v_params, int num_tokens,
                                    int num_kv_heads, int head_dim, int block_size,
                                    int num_blocks, int32_t* error_word,
                                    struct CUstream_st* stream) {
    if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || !plain_dtype(new_dtype))
        return PA_ERR_INVALID_ARG;
    if (head_dim % 32 != 0 || head_dim > pa::kMaxHeadDim || num_kv_heads > kMaxHeads)
        return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!k_new || !v_new || !slot_mapping || !aligned16(k_new) || !aligned16(v_new) ||
        !aligned(slot_mapping, 8) || !pool4_ok(k_cache, v_cache, k_params, v_params))
        return PA_ERR_INVALID_ARG;
    return status_of(pa::launch_append_int4(k_new, v_new, new_dtype, slot_mapping, k_cache,
                                            v_cache, k_params, v_params, num_tokens, num_kv_heads,
                                            head_dim, block_size, num_blocks, error_word,
                                            stream_of(stream)));
}

pa_status pa_gather_int4(const void* k_cache, const void* v_cache, const void* k_params,
                         const void* v_params, const int32_t* block_tables,
                         const int32_t* context_lens, const int64_t* row_starts, void* k_out,
                         void* v_out, pa_dtype out_dtype, int64_t num_rows, int num_seqs,
                         int num_kv_heads, int head_dim, int block_size, int num_blocks,
                         int max_blocks_per_seq, int max_context_len, int32_t* error_word,
                         struct CUstream_st* stream) {
    if (num_seqs < 0 || num_rows < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || max_blocks_per_seq < 0 || max_context_len < 0 || !plain_dtype(out_dtype))
        return PA_ERR_INVALID_ARG;
    if (static_cast<long long>(max_context_len) > static_cast<long long>(max_blocks_per_seq) * block_size)
        return PA_ERR_INVALID_ARG;
    if (head_dim % 32 != 0 || head_dim > pa::kMaxHeadDim || num_kv_heads > kMaxHeads)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    // With no rows to write the outputs may be null; lengths are still checked.
    if (!block_tables || !context_lens || !row_starts || (num_rows > 0 && (!k_out || !v_out)) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(row_starts, 8) ||
        !aligned16(k_out) || !aligned16(v_out) || !pool4_ok(k_cache, v_cache, k_params, v_params))
        return PA_ERR_INVALID_ARG;
    return status_of(pa::launch_gather_int4(k_cache, v_cache, k_params, v_params, block_tables,
                                            context_lens, row_starts, k_out, v_out, out_dtype,
                                            num_rows, num_seqs, num_kv_heads, head_dim, block_size,
                                            num_blocks, max_blocks_per_seq, max_context_len,
                                            error_word, stream_of(stream)));
}

pa_status pa_decode_int4(const void* q, const void* k_cache, const void* v_cache,
                         const void* k_params, const void* v_params, const int32_t* block_tables,
                         const int32_t* context_lens, float scale, int window, void* out,
                         int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                         int head_dim, int block_size, int num_blocks, int max_blocks_per_seq,
                         int max_context_len, void* workspace, size_t workspace_bytes,
                         int32_t* error_word, struct CUstream_st* stream) {
    if (num_seqs < 0 || num_queries < 1 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq < 0 || max_context_len < 0 ||
        window < 0 || num_heads % num_kv_heads != 0 || !std::isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (static_cast<long long>(max_context_len) > static_cast<long long>(max_blocks_per_seq) * block_size)
        return PA_ERR_INVALID_ARG;
    // Row numbers stay below 2^31 with an item's rows added, tile numbers of the
    // pool below 2^32.
    if ((head_dim != 64 && head_dim != 128) || block_size % 16 != 0 ||
        static_cast<long long>(num_heads / num_kv_heads) * num_queries > 8 ||
        max_context_len > INT_MAX - 4096 || num_heads > kMaxHeads ||
        static_cast<double>(num_blocks) * num_kv_heads * (block_size / 16) >= 4294967296.0)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!q || !out || !block_tables || !context_lens || !aligned16(q) || !aligned16(out) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !pool4_ok(k_cache, v_cache, k_params, v_params))
        return PA_ERR_INVALID_ARG;
    // The rows that any of the Q tokens sees: the last window + Q - 1. A window
    // that no row can be outside of is none.
    const int rows_seen =
        (window == 0 || window >= max_context_len) ? 0 : window + num_queries - 1;
    // Partitions of the longest sequence: a windowed one spans its rows seen and
    // up to 15 before them in the same tile. With one there is nothing to merge.
    constexpr int P = pa::kDefaultPartition4;
    const long long most = rows_seen > 0 && rows_seen + 15 < max_context_len ? rows_seen + 15 : max_context_len;
    const long long parts = most > P + pa::kPartitionTail4 ? ceil_div(most - pa::kPartitionTail4, P) : 1;
    const long long chunk = num_seqs < pa::kPlanMaxSeqs ? num_seqs : pa::kPlanMaxSeqs;
    if (parts * chunk * num_kv_heads > 0x3fffffffLL) return PA_ERR_UNSUPPORTED;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < pa_decode_workspace_size_multi(num_seqs, num_queries, num_heads, head_dim,
                                                         max_context_len))
        return PA_ERR_WORKSPACE;

    // The workspace as pa_decode lays it out: 256 bytes, the work items, then
    // the partitions' maxima and sums, then their outputs.
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const size_t units = static_cast<size_t>(chunk) * num_heads * parts;
    pa::DecodeParams base{};
    base.k_cache = k_cache;
    base.v_cache = v_cache;
    base.items = reinterpret_cast<int4*>(ws + 256);
    if (parts > 1) {
        // The outputs are written 16 bytes at a time, so they start on such a
        // boundary: 8 bytes more at most, and the size asked for is for half the
        // partition size.
        base.part_ml = reinterpret_cast<float*>(ws + 256 + 16 * units);
        base.part_o = base.part_ml + (2 * units * num_queries + 3) / 4 * 4;
    }
    base.error_word = error_word;
    base.scale_log2 = scale * kLog2e;
    base.k_scale = base.v_scale = 1.0f;
    base.k_pairs = static_cast<const uint32_t*>(k_params);
    base.v_pairs = static_cast<const uint32_t*>(v_params);
    base.num_queries = num_queries;
    base.window = rows_seen;
    base.num_heads = num_heads;
    base.num_kv_heads = num_kv_heads;
    base.head_dim = head_dim;
    base.block_size = block_size;
    base.num_blocks = num_blocks;
    base.max_blocks_per_seq = max_blocks_per_seq;
    base.context_cap = max_context_len;
    base.partition_size = base.partition_long = P;
    base.partition_long_from = pa::kNoLongPartitions;
    base.partition_tail = pa::kPartitionTail4;
    base.combine_chunk = pa::kCombineChunk4;
    base.max_parts = static_cast<int>(parts);
    // Batches above kPlanMaxSeqs sequences run as consecutive launches over
    // slices of the batch; they reuse the workspace in stream order.
    for (int s0 = 0; s0 < num_seqs; s0 += pa::kPlanMaxSeqs) {
        pa::DecodeParams p = base;
        const size_t qoff = static_cast<size_t>(s0) * num_queries * num_heads * head_dim * 2;
        p.q = static_cast<const uint8_t*>(q) + qoff;
        p.out = static_cast<uint8_t*>(out) + qoff;
        p.block_tables = block_tables + static_cast<size_t>(s0) * max_blocks_per_seq;
        p.context_lens = context_lens + s0;
        p.num_seqs = num_seqs - s0 < pa::kPlanMaxSeqs ? num_seqs - s0 : pa::kPlanMaxSeqs;
        if (pa::launch_decode_int4(p, stream_of(stream)) != cudaSuccess) return PA_ERR_CUDA;
        if (parts > 1 && pa::launch_combine(p, PA_DTYPE_BF16, stream_of(stream)) != cudaSuccess)
            return PA_ERR_CUDA;
    }
    return PA_OK;
}

pa_status pa_norm_rope(const pa_norm_rope_args* args, void* k_out, int64_t k_out_stride,
                       int32_t* error_word, struct CUstream_st* stream) {
    pa::NormRopeParams p{};
    const pa_status ps = norm_rope_params(args, &p);
    if (ps != PA_OK || args->num_tokens == 0) return ps;
    const int64_t unit = 16 / (args->dtype == PA_DTYPE_F32 ? 4 : 2);
    if (!k_out || !aligned16(k_out) || k_out_stride % unit != 0 ||
        k_out_stride < static_cast<int64_t>(args->num_kv_heads) * args->head_dim)
        return PA_ERR_INVALID_ARG;
    p.k_out = k_out;
    p.k_out_stride = k_out_stride;
    p.error_word = error_word;
    return status_of(pa::launch_norm_rope(p, static_cast<pa_dtype>(args->dtype), stream_of(stream)));
}

pa_status pa_norm_rope_append(const pa_norm_rope_args* args, const void* v, int64_t v_stride,
                              const int64_t* slot_mapping, void* k_cache, void* v_cache,
                              int block_size, int num_blocks, int32_t* error_word,
                              struct CUstream_st* stream) {
    pa::NormRopeParams p{};
    pa_status ps = norm_rope_params(args, &p);
    if (ps == PA_OK && (block_size <= 0 || num_blocks <= 0)) ps = PA_ERR_INVALID_ARG;
    if (ps != PA_OK || args->num_tokens == 0) return ps;
    ps = append_params(args, v, v_stride, slot_mapping, block_size, num_blocks, error_word, &p);
    if (ps != PA_OK) return ps;
    if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    return status_of(pa::launch_norm_rope(p, static_cast<pa_dtype>(args->dtype), stream_of(stream)));
}

pa_status pa_norm_rope_append_int4(const pa_norm_rope_args* args, const void* v,
                                   int64_t v_stride, const int64_t* slot_mapping, void* k_cache,
                                   void* v_cache, void* k_params, void* v_params, int block_size,
                                   int num_blocks, int32_t* error_word,
                                   struct CUstream_st* stream) {
    pa::NormRopeParams p{};
    pa_status ps = norm_rope_params(args, &p);
    if (ps == PA_OK && (block_size <= 0 || num_blocks <= 0)) ps = PA_ERR_INVALID_ARG;
    if (ps == PA_OK && args->head_dim % 32 != 0) ps = PA_ERR_UNSUPPORTED;
    if (ps != PA_OK || args->num_tokens == 0) return ps;
    ps = append_params(args, v, v_stride, slot_mapping, block_size, num_blocks, error_word, &p);
    if (ps != PA_OK) return ps;
    if (!pool4_ok(k_cache, v_cache, k_params, v_params)) return PA_ERR_INVALID_ARG;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_params = k_params;
    p.v_params = v_params;
    return status_of(pa::launch_norm_rope(p, static_cast<pa_dtype>(args->dtype), stream_of(stream)));
}

}  // extern "C"
