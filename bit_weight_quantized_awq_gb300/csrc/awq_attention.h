// awq_attention.h -- host-side interface between the tree-attention units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "awq_internal.h"

namespace awq {
namespace attn {

struct Params;

// The kernels' arguments of a call, without its scratch.
Params make_params(const awq_tree_attention_t &a);

// The cache as a 4-D tensor (head_dim, kv_heads, block_size, num_blocks), boxes of 64 elements of
// one head for min(block_size, tile_keys) tokens of one block, 128-byte swizzle.
bool make_cache_map(CUtensorMap *m, const awq_tree_attention_t &a, const awq_cache_t &c, int tile_keys);
bool make_cache_map_5d(CUtensorMap *m, const awq_tree_attention_t &a, const awq_cache_t &c, int tile_keys, int halves);

// The tensor-core kernel (head_dim <= 128), and the partial sums its largest launch keeps.
cudaError_t launch_tc_any(const awq_tree_attention_t &a, cudaStream_t stream);
size_t tc_partial_floats(int sms, int64_t head_dim);

} // namespace attn
} // namespace awq
