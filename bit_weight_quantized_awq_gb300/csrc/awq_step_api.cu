// awq_step_api.cu -- the C ABI of the decoding step around the quantised
// layers (include/awq_gb300.h): argument checks of awq_paged_plan, awq_kv_append,
// awq_rotary, awq_tree_attention, awq_process_logits, awq_beam_select,
// awq_reorder_states and the calls on pages. Nothing aborts and no C++ exception
// leaves an entry point.
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

// What awq_free_pages and awq_compact_pages ask of their sizes.
bool pages_ok(int64_t rows, int64_t width, int64_t stride, int64_t block_size, int64_t num_blocks, int64_t num_held)
{
    return rows >= 0 && rows <= (1 << 20) && width > 0 && width <= kInt / 2 && stride >= width && page_size_ok(block_size) &&
           num_blocks > 0 && num_blocks <= (1 << 28) && num_held >= 0 && num_held < kInt;
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

awq_status_t awq_rotary(const awq_rotary_t *args, awq_stream_t stream)
{
    if (!args) return AWQ_ERR_INVALID_ARG;
    const awq_rotary_t &a = *args;
    const bool append = a.slot_map != nullptr;
    if ((a.dtype != AWQ_F16 && a.dtype != AWQ_BF16) || a.tokens < 0 || a.tokens >= kInt || a.q_heads <= 0 ||
        a.kv_heads < 0 || (append && a.kv_heads == 0) || a.q_heads >= (1 << 24) || a.kv_heads >= (1 << 24) ||
        a.head_dim <= 0 || a.head_dim % 8 != 0 || a.head_dim > 1024 ||
        (a.q_heads + 2 * a.kv_heads) * a.head_dim >= (1 << 24) || a.rotary_dim <= 0 || a.rotary_dim % 2 != 0 ||
        a.rotary_dim > a.head_dim || a.num_axes < 1 || a.num_axes >= kInt)
        return AWQ_ERR_INVALID_ARG;
    const int64_t strides[] = {a.q_token_stride, a.q_head_stride, a.k_token_stride, a.k_head_stride,
                               a.v_token_stride, a.v_head_stride, a.q_out_token_stride, a.q_out_head_stride,
                               a.k_out_token_stride, a.k_out_head_stride};
    for (const int64_t s : strides)
        if (s < 0 || s % 8 != 0 || s >= (int64_t(1) << 38)) return AWQ_ERR_INVALID_ARG;
    if (append && (!page_size_ok(a.block_size) || a.num_blocks < 0 || a.num_blocks >= kInt ||
                   !cache_strides_ok(a.k_cache) || !cache_strides_ok(a.v_cache)))
        return AWQ_ERR_INVALID_ARG;
    if ((a.q_out == a.q && (a.q_out_token_stride != a.q_token_stride || a.q_out_head_stride != a.q_head_stride)) ||
        (!append && a.k && a.k_out == a.k &&
         (a.k_out_token_stride != a.k_token_stride || a.k_out_head_stride != a.k_head_stride)))
        return a.tokens == 0 ? AWQ_OK : AWQ_ERR_INVALID_ARG;
    if (a.tokens == 0) return AWQ_OK;
    if (!a.q || !a.q_out || !a.positions || !a.inv_freq || (a.kv_heads > 0 && !a.k) ||
        (append ? !a.v || !a.k_cache.data || !a.v_cache.data : a.kv_heads > 0 && !a.k_out))
        return AWQ_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.q_out, 16) || !aligned(a.k_out, 16) ||
        !aligned(a.positions, 4) || !aligned(a.inv_freq, 4) || !aligned(a.axes, 4) || !aligned(a.slot_map, 8) ||
        (append && (!aligned(a.k_cache.data, 16) || !aligned(a.v_cache.data, 16))))
        return AWQ_ERR_MISALIGNED;
    return launched([&] { return awq::launch_rotary(a, reinterpret_cast<cudaStream_t>(stream)); });
}

int64_t awq_beam_select_workspace(int64_t requests, int64_t beams, int64_t vocab, int64_t num_beams, int64_t num_ends,
                                  awq_dtype_t dtype)
{
    if (requests < 0 || requests > kMaxRequests || beams < 1 || beams > 32 || num_beams < 1 || num_beams > 32 ||
        num_ends < 0 || num_ends > 8 || vocab <= 0 || vocab > (int64_t(1) << 27) ||
        (dtype != AWQ_F16 && dtype != AWQ_BF16 && dtype != AWQ_F32))
        return -1;
    const int64_t best = num_beams + num_ends;
    return 8 * awq::beam_cut(requests, beams, vocab, best, dtype == AWQ_F32 ? 4 : 2).words;
}

awq_status_t awq_beam_select(const awq_beam_select_t *args, awq_stream_t stream)
{
    if (!args) return AWQ_ERR_INVALID_ARG;
    const awq_beam_select_t &a = *args;
    const int64_t bytes =
        awq_beam_select_workspace(a.requests, a.beams, a.vocab, a.num_beams, a.num_ends, (awq_dtype_t)a.dtype);
    if (bytes < 0 || (a.num_ends > 0 && !a.end_tokens)) return AWQ_ERR_INVALID_ARG;
    if (a.requests * a.beams > 1 && (a.logits_row_stride < a.vocab || a.logits_row_stride >= int64_t(1) << 38))
        return AWQ_ERR_INVALID_ARG;
    if (a.requests == 0) return AWQ_OK;
    if (!a.logits || !a.scores || !a.out_scores || !a.out_parents || !a.out_tokens || !a.workspace ||
        a.workspace_bytes < bytes || ((a.num_ends > 0 || a.ended_scores) && (!a.ended_scores || !a.ended_parents || !a.ended_tokens)))
        return AWQ_ERR_INVALID_ARG;
    if (!aligned(a.logits, a.dtype == AWQ_F32 ? 4 : 2) || !aligned(a.scores, 4) || !aligned(a.end_tokens, 4) ||
        !aligned(a.out_scores, 4) || !aligned(a.out_parents, 4) || !aligned(a.out_tokens, 4) ||
        !aligned(a.ended_scores, 4) || !aligned(a.ended_parents, 4) || !aligned(a.ended_tokens, 4) ||
        !aligned(a.workspace, 256))
        return AWQ_ERR_MISALIGNED;
    return launched([&] { return awq::launch_beam_select(a, reinterpret_cast<cudaStream_t>(stream)); });
}

awq_status_t awq_reorder_states(const awq_state_t *states, int64_t count, const int32_t *parents, int64_t rows_out,
                                int64_t rows_in, awq_stream_t stream)
{
    if (count < 0 || count > 4096 || rows_out < 0 || rows_out >= kInt || rows_in < 0 || rows_in >= kInt ||
        (count > 0 && !states))
        return AWQ_ERR_INVALID_ARG;
    for (int64_t i = 0; i < count; ++i) {
        const awq_state_t &s = states[i];
        if (s.row_bytes < 0 || s.row_bytes >= kInt || s.src_row_stride >= (int64_t(1) << 40) ||
            s.dst_row_stride >= (int64_t(1) << 40) || (rows_in > 1 && s.src_row_stride < s.row_bytes) ||
            (rows_out > 1 && s.dst_row_stride < s.row_bytes) ||
            (rows_out > 0 && s.row_bytes > 0 && (!s.dst || (rows_in > 0 && !s.src))))
            return AWQ_ERR_INVALID_ARG;
    }
    if (count == 0 || rows_out == 0) return AWQ_OK;
    if (!parents) return AWQ_ERR_INVALID_ARG;
    if (!aligned(parents, 4)) return AWQ_ERR_MISALIGNED;
    return launched([&] {
        return awq::launch_reorder_states(states, count, parents, rows_out, rows_in,
                                          reinterpret_cast<cudaStream_t>(stream));
    });
}

awq_status_t awq_fork_pages(const int32_t *block_table, int64_t rows_in, int64_t table_width, int64_t table_stride,
                            const int32_t *lens, const int32_t *parents, int64_t rows_out, const int32_t *free_blocks,
                            int64_t num_free, const int32_t *free_start, int64_t block_size, int32_t *new_table,
                            int64_t new_stride, int32_t *new_lens, int32_t *src, int32_t *dst, int32_t *tokens,
                            int32_t *count, awq_stream_t stream)
{
    if (rows_in < 0 || rows_in > kMaxRequests || rows_out < 0 || rows_out > kMaxRequests || !page_size_ok(block_size) ||
        table_width <= 0 || table_width > kInt / 2 || table_stride < table_width || new_stride < table_width ||
        num_free < 0 || num_free >= kInt)
        return AWQ_ERR_INVALID_ARG;
    if (!count || (rows_in > 0 && (!block_table || !lens)) || (num_free > 0 && !free_blocks) ||
        (rows_out > 0 && (!parents || !new_table || !new_lens || !src || !dst || !tokens)) ||
        (rows_in > 0 && rows_out > 0 && new_table == block_table))
        return AWQ_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(lens, 4) || !aligned(parents, 4) || !aligned(free_blocks, 4) ||
        !aligned(free_start, 4) || !aligned(new_table, 4) || !aligned(new_lens, 4) || !aligned(src, 4) ||
        !aligned(dst, 4) || !aligned(tokens, 4) || !aligned(count, 4))
        return AWQ_ERR_MISALIGNED;
    const awq::ForkProblem p{block_table, lens, parents, free_blocks, free_start, new_table, new_lens, src, dst, tokens,
                             count, table_stride, new_stride, (int)rows_in, (int)rows_out, (int)table_width,
                             (int)num_free, (int)block_size};
    return launched([&] { return awq::launch_fork_pages(p, reinterpret_cast<cudaStream_t>(stream)); });
}

awq_status_t awq_copy_pages(void *const *caches, int64_t num_caches, const awq_cache_t *layout, int64_t num_blocks,
                            int64_t block_size, int64_t kv_heads, int64_t head_dim, const int32_t *src,
                            const int32_t *dst, const int32_t *tokens, int64_t pairs, const int32_t *count,
                            awq_stream_t stream)
{
    if (num_caches < 0 || num_caches > 65536 || pairs < 0 || pairs >= kInt || num_blocks <= 0 || num_blocks >= kInt ||
        !page_size_ok(block_size) || kv_heads <= 0 || head_dim <= 0 || head_dim % 8 != 0 || kv_heads >= (1 << 20) ||
        head_dim >= (1 << 20) || kv_heads * head_dim * block_size >= (int64_t(1) << 30) || !layout ||
        !cache_strides_ok(*layout))
        return AWQ_ERR_INVALID_ARG;
    if (num_caches == 0 || pairs == 0) return AWQ_OK;
    if (!caches || !src || !dst) return AWQ_ERR_INVALID_ARG;
    for (int64_t i = 0; i < num_caches; ++i) {
        if (!caches[i]) return AWQ_ERR_INVALID_ARG;
        if (!aligned(caches[i], 16)) return AWQ_ERR_MISALIGNED;
    }
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(tokens, 4) || !aligned(count, 4)) return AWQ_ERR_MISALIGNED;
    const awq::CopyProblem p{caches, *layout, src, dst, tokens, count, num_caches, pairs, (int)num_blocks,
                             (int)block_size, (int)kv_heads, (int)head_dim};
    return launched([&] { return awq::launch_copy_pages(p, reinterpret_cast<cudaStream_t>(stream)); });
}

int64_t awq_pages_workspace(int64_t num_blocks)
{
    if (num_blocks <= 0 || num_blocks > (int64_t(1) << 28)) return -1;
    const int64_t words = (num_blocks + 31) / 32;      // the bitmap, sums before its words, sums of 256 words
    return 8 * words + (words + 255) / 256 * 4 + 16;
}

awq_status_t awq_free_pages(const int32_t *block_table, int64_t rows, int64_t table_width, int64_t table_stride,
                            const int32_t *lens, int64_t block_size, int64_t num_blocks, const int32_t *held,
                            int64_t num_held, int32_t *free_blocks, int32_t *counts, void *workspace,
                            awq_stream_t stream)
{
    if (!pages_ok(rows, table_width, table_stride, block_size, num_blocks, num_held) || !free_blocks || !counts ||
        !workspace || (rows > 0 && (!block_table || !lens)) || (num_held > 0 && !held))
        return AWQ_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(lens, 4) || !aligned(held, 4) || !aligned(free_blocks, 4) ||
        !aligned(counts, 4) || !aligned(workspace, 256))
        return AWQ_ERR_MISALIGNED;
    awq::PagesProblem p{};
    p.table = block_table;
    p.lens = lens;
    p.held = held;
    p.free_blocks = free_blocks;
    p.counts = counts;
    p.workspace = static_cast<uint32_t *>(workspace);
    p.stride = table_stride;
    p.num_held = num_held;
    p.rows = (int)rows;
    p.width = (int)table_width;
    p.block_size = (int)block_size;
    p.num_blocks = (int)num_blocks;
    return launched([&] { return awq::launch_pages(p, reinterpret_cast<cudaStream_t>(stream)); });
}

awq_status_t awq_compact_pages(const int32_t *block_table, int64_t rows, int64_t table_width, int64_t table_stride,
                               const int32_t *lens, int64_t block_size, int64_t num_blocks, const int32_t *held,
                               int64_t num_held, int32_t *new_table, int64_t new_stride, int32_t *block_map,
                               int32_t *src, int32_t *dst, int32_t *count, void *workspace, awq_stream_t stream)
{
    if (!pages_ok(rows, table_width, table_stride, block_size, num_blocks, num_held) || new_stride < table_width ||
        !block_map || !count || !workspace || (num_blocks > 1 && (!src || !dst)) ||
        (rows > 0 && (!block_table || !lens || !new_table || new_table == block_table)) || (num_held > 0 && !held))
        return AWQ_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(lens, 4) || !aligned(held, 4) || !aligned(new_table, 4) ||
        !aligned(block_map, 4) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(count, 4) || !aligned(workspace, 256))
        return AWQ_ERR_MISALIGNED;
    awq::PagesProblem p{};
    p.table = block_table;
    p.lens = lens;
    p.held = held;
    p.new_table = new_table;
    p.block_map = block_map;
    p.src = src;
    p.dst = dst;
    p.moves = count;
    p.workspace = static_cast<uint32_t *>(workspace);
    p.stride = table_stride;
    p.new_stride = new_stride;
    p.num_held = num_held;
    p.rows = (int)rows;
    p.width = (int)table_width;
    p.block_size = (int)block_size;
    p.num_blocks = (int)num_blocks;
    return launched([&] { return awq::launch_pages(p, reinterpret_cast<cudaStream_t>(stream)); });
}

} // extern "C"
