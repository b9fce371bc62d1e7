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

} // namespace attn
} // namespace awq
