// awq_step_api.cu -- the C ABI of the decoding step around the quantised
// layers (include/awq_gb300.h): argument checks of awq_paged_plan,
// awq_kv_append, awq_tree_attention and awq_process_logits. Nothing aborts and
// no C++ exception leaves an entry point.
#include <cstdint>

#include <cuda_runtime.h>

#include "awq_internal.h"

namespace {

using awq::kMaxRequests;
constexpr int64_t kInt = int64_t(1) << 31;   // sizes below this fit an int

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool page_size_ok(int64_t n) { return n >= 16 && n <= 1024 && (n & (n - 1)) == 0; }

// Strides in elements of 2 bytes that keep every row on a 16-byte boundary.
bool cache_strides_ok(const awq_cache_t &c)
{
    constexpr int64_t most = int64_t(1) << 38;   // elements: a tensor map's strides stay below 2^40 bytes
    return c.block_stride > 0 && c.token_stride > 0 && c.head_stride > 0 && c.block_stride < most &&
           c.token_stride < most && c.head_stride < most && c.block_stride % 8 == 0 && c.token_stride % 8 == 0 &&
           c.head_stride % 8 == 0;
}

template <typename F>
awq_status_t launched(F launch)
{
    try {
        const cudaError_t e = launch();
        if (e == cudaSuccess) return AWQ_OK;
        if (awq::scratch_over_reservation()) {
            awq::clear_scratch_over_reservation();
            return AWQ_ERR_TOO_LARGE;
        }
    } catch (...) {
    }
    return AWQ_ERR_CUDA;
}

} // namespace

extern "C" {

awq_status_t awq_paged_plan(const int32_t *context_lens, const int32_t *new_lens, int64_t B, int32_t *block_table,
                            int64_t table_width, int64_t table_stride, const int32_t *free_blocks, int64_t num_free,
                            int64_t block_size, const int32_t *parents, int64_t max_tokens, int32_t *cu_new,
                            int64_t *slot_map, int32_t *positions, int32_t *token_request, int32_t *tree_mask,
                            int64_t mask_words, int32_t *counts, awq_stream_t stream)
{
    if (B < 0 || B > kMaxRequests || !page_size_ok(block_size) || max_tokens < 0 || max_tokens > (int64_t(1) << 30) ||
        table_width <= 0 || table_width >= kInt || table_stride < table_width || num_free < 0 || num_free >= kInt ||
        mask_words < 0 || mask_words > 1024)
        return AWQ_ERR_INVALID_ARG;
    if (!cu_new || !counts || (B > 0 && (!context_lens || !new_lens || !block_table)) ||
        (num_free > 0 && !free_blocks) || (max_tokens > 0 && (!slot_map || !positions || !token_request)) ||
        (max_tokens > 0 && mask_words > 0 && !tree_mask))
        return AWQ_ERR_INVALID_ARG;
    if (!aligned(context_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(free_blocks, 4) ||
        !aligned(parents, 4) || !aligned(cu_new, 4) || !aligned(slot_map, 8) || !aligned(positions, 4) ||
        !aligned(token_request, 4) || !aligned(tree_mask, 4) || !aligned(counts, 4))
        return AWQ_ERR_MISALIGNED;
    awq::PlanProblem p{context_lens, new_lens, block_table, free_blocks, parents, cu_new, slot_map, positions,
                       token_request, tree_mask, counts, table_stride, (int)B, (int)table_width, (int)num_free,
                       (int)block_size, (int)max_tokens, (int)mask_words};
    return launched([&] { return awq::launch_paged_plan(p, reinterpret_cast<cudaStream_t>(stream)); });
}

awq_status_t awq_kv_append(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                           int64_t v_token_stride, int64_t v_head_stride, const awq_cache_t *k_cache,
                           const awq_cache_t *v_cache, const int64_t *slot_map, int64_t tokens, int64_t num_blocks,
                           int64_t block_size, int64_t kv_heads, int64_t head_dim, awq_stream_t stream)
{
    if (tokens < 0 || tokens >= kInt || num_blocks < 0 || num_blocks >= kInt || !page_size_ok(block_size) ||
        kv_heads <= 0 || head_dim <= 0 || head_dim % 8 != 0 || kv_heads >= (1 << 20) || head_dim >= (1 << 20) ||
        kv_heads * head_dim >= (int64_t(1) << 24) || !k_cache || !v_cache)
        return AWQ_ERR_INVALID_ARG;
    if (k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 || v_head_stride % 8 || k_token_stride < 0 ||
        k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0 || !cache_strides_ok(*k_cache) ||
        !cache_strides_ok(*v_cache))
        return AWQ_ERR_INVALID_ARG;
    if (tokens == 0) return AWQ_OK;
    if (!k || !v || !k_cache->data || !v_cache->data || !slot_map) return AWQ_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache->data, 16) || !aligned(v_cache->data, 16) ||
        !aligned(slot_map, 8))
        return AWQ_ERR_MISALIGNED;
    awq::AppendProblem p{k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride, *k_cache, *v_cache,
                         slot_map, tokens, num_blocks, (int)block_size, (int)kv_heads, (int)head_dim};
    return launched([&] { return awq::launch_kv_append(p, reinterpret_cast<cudaStream_t>(stream)); });
}

awq_status_t awq_tree_attention(const awq_tree_attention_t *args, awq_stream_t stream)
{
    if (!args) return AWQ_ERR_INVALID_ARG;
    const awq_tree_attention_t &a = *args;
    if (a.dtype != AWQ_F16 && a.dtype != AWQ_BF16) return AWQ_ERR_INVALID_ARG;
    if (a.B < 0 || a.B > kMaxRequests || a.tokens < 0 || a.tokens >= kInt || a.q_heads <= 0 || a.kv_heads <= 0 ||
        a.q_heads >= kInt || a.q_heads % a.kv_heads != 0 || a.tokens * a.q_heads >= kInt - 1024 || a.head_dim <= 0 ||
        a.head_dim % 8 != 0 || a.head_dim > 256 || a.num_blocks <= 0 || a.num_blocks >= kInt ||
        !page_size_ok(a.block_size) || a.max_new < 0 || a.max_context < 0 || a.max_new >= kInt || a.max_context >= kInt)
        return AWQ_ERR_INVALID_ARG;
    if (a.table_width <= 0 || a.table_stride < a.table_width || a.table_width * a.block_size >= kInt - 1024 ||
        a.table_width >= kInt || (a.tree_mask && (a.mask_words <= 0 || a.mask_words > (1 << 20))))
        return AWQ_ERR_INVALID_ARG;
    if (a.q_token_stride % 8 || a.q_head_stride % 8 || a.q_token_stride < 0 || a.q_head_stride < 0 ||
        !cache_strides_ok(a.k_cache) || !cache_strides_ok(a.v_cache))
        return AWQ_ERR_INVALID_ARG;
    if (a.tokens == 0 || a.B == 0) return AWQ_OK;
    if (!a.q || !a.out || !a.k_cache.data || !a.v_cache.data || !a.block_table || !a.context_lens || !a.cu_new)
        return AWQ_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.k_cache.data, 16) || !aligned(a.v_cache.data, 16) ||
        !aligned(a.lse, 4) || !aligned(a.block_table, 4) || !aligned(a.context_lens, 4) || !aligned(a.cu_new, 4) ||
        !aligned(a.tree_mask, 4))
        return AWQ_ERR_MISALIGNED;
    return launched([&] { return awq::launch_tree_attention(a, reinterpret_cast<cudaStream_t>(stream)); });
}

awq_status_t awq_process_logits(const awq_logits_t *args, awq_stream_t stream)
{
    if (!args) return AWQ_ERR_INVALID_ARG;
    const awq_logits_t &a = *args;
    const uintptr_t size = a.dtype == AWQ_F32 ? 4 : 2;
    if (a.dtype != AWQ_F16 && a.dtype != AWQ_BF16 && a.dtype != AWQ_F32) return AWQ_ERR_INVALID_ARG;
    if (a.rows < 0 || a.rows >= kInt || a.vocab <= 0 || a.vocab > (int64_t(1) << 27) || a.B < 0 || a.B >= kInt ||
        a.history_size < 0 || a.history_size >= (int64_t(1) << 29) || a.bias_size < 0 || a.bias_size > kInt / 2 || a.mask_words < 0 ||
        a.mask_words > (1 << 20) || a.grammar_count < 0)
        return AWQ_ERR_INVALID_ARG;
    if (a.rows > 1 && (a.logits_row_stride < a.vocab || a.out_row_stride < a.vocab)) return AWQ_ERR_INVALID_ARG;
    if ((a.history && !a.history_offsets) || (a.draft_tokens && !a.cu_new) ||
        (a.tree_mask && a.draft_tokens && a.mask_words == 0) ||
        ((a.bias_tokens != nullptr) != (a.bias_values != nullptr)) || (a.bias_tokens && !a.bias_offsets) ||
        (a.out == a.logits && a.rows > 1 && a.out_row_stride != a.logits_row_stride))
        return AWQ_ERR_INVALID_ARG;
    if (a.rows == 0) return AWQ_OK;
    if (!a.logits || !a.out) return AWQ_ERR_INVALID_ARG;
    if (!aligned(a.logits, size) || !aligned(a.out, size) || !aligned(a.row_request, 4) || !aligned(a.history, 4) ||
        !aligned(a.history_offsets, 4) || !aligned(a.prompt_lens, 4) || !aligned(a.repetition, 4) ||
        !aligned(a.frequency, 4) || !aligned(a.presence, 4) || !aligned(a.draft_tokens, 4) || !aligned(a.cu_new, 4) ||
        !aligned(a.tree_mask, 4) || !aligned(a.bias_tokens, 4) || !aligned(a.bias_offsets, 4) ||
        !aligned(a.bias_values, 4) || !aligned(a.grammar_mask, 4) || !aligned(a.grammar_rows, 4))
        return AWQ_ERR_MISALIGNED;
    return launched([&] { return awq::launch_process_logits(a, reinterpret_cast<cudaStream_t>(stream)); });
}

} // extern "C"
