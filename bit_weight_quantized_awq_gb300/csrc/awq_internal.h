// awq_internal.h -- host-side interface between the C-ABI layer (awq_api.cu)
// and the kernel translation units. Not installed; not part of the ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/awq_gb300.h"

namespace awq {

// One validated forward/dequant problem. g is the resolved group size (the
// page's group_size -1 already replaced by K), G = K / g.
struct Problem {
    const void *x;          // fp16 [M, K]
    const int32_t *qweight; // int32 [K, N / 8]
    const int32_t *qzeros;  // int32 [G, N / 8]
    const void *scales;     // fp16 [G, N]
    const void *bias;       // fp16 [N] or nullptr
    void *y;                // fp16 [M, N]
    int64_t M, K, N, g, G;
    int64_t ldx = 0;        // elements between rows of x (0 = K): a K-slice of a wider x
    float *y32 = nullptr;   // if set: y32[M, N] += x . W in fp32 (no bias, no rounding),
                            // instead of writing y
    const int32_t *row_perm = nullptr;   // dequantise-then-GEMM only: weight row k is
                                         // row row_perm[k] of W (act-order layers)
};

// Per-(device, stream) scratch: fp32 split-K partials plus self-resetting
// per-tile arrival counters (zero between calls).
struct Scratch {
    float *partials;
    size_t partial_floats;
    unsigned int *counters;
    size_t n_counters;
};

// Bumped by awq_shutdown(): per-device values a launcher caches (symbol
// addresses, function attributes set once per device) are looked up again
// when the generation they were cached in is no longer current.
unsigned cache_generation();

#ifdef AWQ_FAULT_TEST
// Fault-test build only: when non-zero, the next decode and prefill launches
// tell CTA 0's TMA producer to issue nothing, so that the waits of that CTA's
// consumers on the stage barriers run out (see awq_gb300_fault_test.h).
int fault_injection();
#endif

// Returns the address of this device's status word (bit flags, see
// kStatusTimeout) for kernels to record device-side errors in.
unsigned int *device_status_word();
constexpr unsigned int kStatusTimeout = 1u;
constexpr unsigned int kStatusBadIndex = 2u;   // a group or row index out of range
constexpr unsigned int kStatusTooLarge = 4u;   // a capacity exceeded (free blocks, table width, tokens)

// Scratch for `stream` on the current device, grown to at least the given
// sizes. Returns false if an allocation failed, or if the stream's scratch
// was reserved (awq_reserve) and is smaller than asked: a reserved area never
// grows (scratch_over_reservation() then reports true on this thread).
bool get_scratch(cudaStream_t stream, size_t partial_floats, size_t n_counters, Scratch *out);
bool scratch_over_reservation();
void clear_scratch_over_reservation();

// Largest split-K partial areas (floats) a decode / prefill launch on a GPU
// with `sms` SMs asks for, whatever the shape.
size_t decode_partial_floats_max(int sms);
size_t prefill_partial_floats_max(int sms);

// A buffer of at least `bytes` for `stream` on the current device (dequantised
// weights of the g_idx forward), grown on demand.
bool get_w16_scratch(cudaStream_t stream, size_t bytes, void **out);

// ---- kernel launchers (each returns the launch's cudaError_t) ----

cudaError_t launch_dequant(const Problem &p, void *W, cudaStream_t stream);

// Dequantisation of output columns c0 .. c0 + nc - 1 (multiples of 8) into a
// [K, nc] fp16 array.
cudaError_t launch_dequant_cols(const Problem &p, int64_t c0, int64_t nc, void *W, cudaStream_t stream);

// Large-M forward: the weights dequantised once per column window into a
// per-stream scratch area, then the tcgen05 fp16 GEMM core on each window.
cudaError_t launch_dequant_gemm(const Problem &p, cudaStream_t stream);

// Dequantisation with the group of row k taken from g_idx[k] (p.G groups);
// an index outside [0, G) writes zeros for that row and sets kStatusBadIndex.
cudaError_t launch_dequant_gidx(const Problem &p, const int32_t *g_idx, void *W, cudaStream_t stream);

// y[M, N] = fp16_rn(y32 + bias): the end of a row-parallel forward.
cudaError_t launch_finish_rows(const float *y32, const void *bias, void *y, int64_t M, int64_t N,
                               cudaStream_t stream);

// Packing of 4-bit codes (uint8, one per byte) into int32 words, and
// round-to-nearest quantisation of an fp16 W with the problem's scales and
// zero points into its qweight.
cudaError_t launch_pack(const uint8_t *codes, int32_t *packed, int64_t rows, int64_t cols,
                        cudaStream_t stream);
cudaError_t launch_quantize(const Problem &p, const void *W, int32_t *qweight, cudaStream_t stream);

cudaError_t launch_generic(const Problem &p, cudaStream_t stream);

// Decode path (small M). supported_* is host-only shape logic.
bool decode_supported(int64_t M, int64_t K, int64_t N, int64_t g);
// columns per decode tile for this shape (0 if the decode kernel cannot serve it)
int decode_tile_columns(int64_t M, int64_t K, int64_t N, int64_t g);
cudaError_t launch_decode(const Problem &p, cudaStream_t stream);

// Prefill path (large M, tcgen05).
bool prefill_supported(int64_t M, int64_t K, int64_t N, int64_t g);
cudaError_t launch_prefill(const Problem &p, cudaStream_t stream);

// The prefill kernel's tensor-core pipeline on an already dequantised fp16
// W [K, N] (no dequant stage): y = x . W + bias. Same shape rules as prefill.
// ldy: elements between rows of y (0 = N), so that a call can write a
// column window of a wider output.
cudaError_t launch_gemm_f16(const Problem &p, const void *w16, cudaStream_t stream, int64_t ldy = 0);
// kernels one prefill / GEMM-core launch enqueues on a GPU with `sms` SMs:
// the persistent kernel, plus sk_fixup_kernel when a tile is split along k
int prefill_launches(int64_t M, int64_t K, int64_t N, int sms);
// act-order layers: rows of packed weights / columns of x in sorted order
cudaError_t launch_gather_rows(const int32_t *src, const int32_t *perm, int32_t *dst, int64_t K,
                               int64_t words, cudaStream_t stream);
cudaError_t launch_gather_cols(const void *x, int64_t ldx, const int32_t *perm, void *xs, int64_t M,
                               int64_t K, cudaStream_t stream);
bool get_xs_scratch(cudaStream_t stream, size_t bytes, void **out);
// ---- the decoding step around the layers (arguments already checked) ----

constexpr int64_t kMaxRequests = 16384;   // of a step

struct PlanProblem {
    const int32_t *context_lens, *new_lens;
    int32_t *block_table;
    const int32_t *free_blocks, *parents;
    int32_t *cu_new;
    int64_t *slot_map;
    int32_t *positions, *token_request, *tree_mask, *counts;
    int64_t table_stride;
    int B, table_width, num_free, block_size, max_tokens, mask_words;
};
cudaError_t launch_paged_plan(const PlanProblem &p, cudaStream_t stream);

struct AppendProblem {
    const void *k, *v;
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    awq_cache_t k_cache, v_cache;
    const int64_t *slot_map;
    int64_t tokens, num_blocks;
    int block_size, kv_heads, head_dim;
};
cudaError_t launch_kv_append(const AppendProblem &p, cudaStream_t stream);

cudaError_t launch_tree_attention(const awq_tree_attention_t &a, cudaStream_t stream);
// floats of partial sums that the largest tree-attention launch of this head_dim or a smaller
// one asks for, whatever the lengths
size_t tree_attention_partial_floats(int64_t head_dim, int sms);

cudaError_t launch_process_logits(const awq_logits_t &a, cudaStream_t stream);

cudaError_t launch_rotary(const awq_rotary_t &a, cudaStream_t stream);

// How beam_select's rows are shared out over CTAs, and its workspace in words of 8 bytes.
struct BeamCut {
    int64_t chunks, chunk, own, span, each, ctas, merge_lists, words;
};
BeamCut beam_cut(int64_t requests, int64_t beams, int64_t vocab, int64_t best, int element_bytes);
cudaError_t launch_beam_select(const awq_beam_select_t &a, cudaStream_t stream);

cudaError_t launch_reorder_states(const awq_state_t *states, int64_t count, const int32_t *parents, int64_t rows_out,
                                  int64_t rows_in, cudaStream_t stream);

struct ForkProblem {
    const int32_t *table, *lens, *parents, *free_blocks, *free_start;
    int32_t *new_table, *new_lens, *src, *dst, *tokens, *count;
    int64_t stride, new_stride;
    int rows_in, rows_out, width, num_free, block_size;
};
cudaError_t launch_fork_pages(const ForkProblem &p, cudaStream_t stream);

struct CopyProblem {
    void *const *caches;
    awq_cache_t layout;
    const int32_t *src, *dst, *tokens, *count;
    int64_t num_caches, pairs;
    int num_blocks, block_size, kv_heads, head_dim;
};
cudaError_t launch_copy_pages(const CopyProblem &p, cudaStream_t stream);

// Of awq_free_pages (free_blocks is set) and of awq_compact_pages.
struct PagesProblem {
    const int32_t *table, *lens, *held;
    int32_t *free_blocks, *counts;
    int32_t *new_table, *block_map, *src, *dst, *moves;
    uint32_t *workspace;          // bit b % 32 of word b / 32: block b is used
    int *prefix, *groups;         // behind it: used blocks before each word, and of each group of words
    int64_t stride, new_stride, num_held;
    int rows, width, block_size, num_blocks;
};
cudaError_t launch_pages(const PagesProblem &p, cudaStream_t stream);

// Allows a kernel this much dynamic shared memory on the current device, once: a limit of a
// call's own size could be lowered by another thread's call before this one's launch.
cudaError_t allow_shared(const void *kernel, size_t bytes);

// A launch whose grid may be scheduled before the kernel ahead of it in the stream has
// ended; the kernel waits for it by itself (ptx::wait_prerequisites). cluster: CTAs of a cluster.
inline cudaError_t launch_dependent(const void *kernel, int64_t grid, int block, size_t smem, cudaStream_t stream,
                                    void **args, int cluster = 1)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// fp16 weight columns per window of the dequantise-then-GEMM path
int64_t dequant_gemm_window(int64_t K, int64_t N);

} // namespace awq
