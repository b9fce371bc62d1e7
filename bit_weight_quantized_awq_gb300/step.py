"""Torch-facing functions of the decoding step around the quantised layers
(``include/awq_gb300.h`` has the operators' definitions). No arithmetic happens
here, nothing waits for the GPU, and what is known on the device only (lengths,
table entries, tokens) is checked there: ``awq_last_device_status`` reports it. The
tensors must be on the current CUDA device (``torch.cuda.set_device``), else ValueError.

A step is ``paged_plan`` -> per layer ``kv_append``, ``tree_attention`` ->
``process_logits``: the plan's ``cu_new``, ``slot_map`` and ``tree_mask`` are the
others' arguments.

The arguments are tested, outputs allocated and the C ABI called in a native module
(``csrc/awq_step_module.cpp``), since a step's kernels take a few microseconds each.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple

import torch

from ._binding import STEP_PATH, AWQError, load_library

_step = None     # the native module, once loaded


def _load():
    """Loads the native module and gives it the library's entry points."""
    global _step
    if not os.path.exists(STEP_PATH):
        raise RuntimeError(f"AWQ step module not found at {STEP_PATH}; build it with "
                           "`python -m bit_weight_quantized_awq_gb300.build`")
    loader = importlib.machinery.ExtensionFileLoader("awq_step", STEP_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("awq_step", STEP_PATH, loader=loader))
    loader.exec_module(module)
    lib = load_library()
    module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in
                  (lib.awq_paged_plan, lib.awq_kv_append, lib.awq_tree_attention, lib.awq_process_logits)))
    _step = module
    return module


class PagedPlan(NamedTuple):
    """What ``paged_plan`` lays out for a step (all on the device, in one allocation)."""
    cu_new: torch.Tensor          # int32 [B + 1]
    slot_map: torch.Tensor        # int64 [max_tokens]
    positions: torch.Tensor       # int32 [max_tokens]
    token_request: torch.Tensor   # int32 [max_tokens]
    tree_mask: torch.Tensor | None    # int32 [max_tokens, mask_words]
    counts: torch.Tensor          # int32 [2]: new tokens, blocks taken from free_blocks


def paged_plan(context_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
               free_blocks: torch.Tensor, block_size: int, max_tokens: int,
               parents: torch.Tensor | None = None, mask_words: int = 0) -> PagedPlan:
    """One step's layout from request lengths: extends ``block_table`` in place
    with blocks from the start of ``free_blocks`` and gives every new token its
    cache slot, position and request, and with ``mask_words`` > 0 its ancestors in
    the drafted tree that ``parents`` describes (a chain if None)."""
    made = (_step or _load()).paged_plan(context_lens, new_lens, block_table, free_blocks, block_size, max_tokens,
                                         parents, mask_words)
    if type(made) is int:
        raise AWQError(made, "awq_paged_plan")
    return PagedPlan._make(made)


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              slot_map: torch.Tensor) -> None:
    """Writes the new tokens' keys and values [tokens, kv_heads, head_dim] (views of
    a fused projection's output serve as they are) into the slots of a paged
    cache [blocks, block_size, kv_heads, head_dim]; slot -1 is skipped."""
    status = (_step or _load()).kv_append(k, v, k_cache, v_cache, slot_map)
    if status is not None:
        raise AWQError(status, "awq_kv_append")


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                   context_lens: torch.Tensor, cu_new: torch.Tensor, scale: float, max_new: int, max_context: int,
                   tree_mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None) -> torch.Tensor:
    """softmax(scale q k^T) v of new tokens [tokens, q_heads, head_dim] over their
    requests' caches, their own keys and values included: a token sees its whole
    context and, of the new tokens, those of its ``tree_mask`` row (itself and
    the ones before it if None). ``max_new`` and ``max_context`` bound the
    lengths; ``lse`` (fp32 [tokens, q_heads]) receives the log-sum-exp. Rows of q past
    ``cu_new``'s end (a plan's padding) are left as they are in ``out``: undefined
    where the call makes it."""
    made = (_step or _load()).tree_attention(q, k_cache, v_cache, block_table, context_lens, cu_new, scale, max_new,
                                             max_context, tree_mask, out, lse)
    if type(made) is int:
        raise AWQError(made, "awq_tree_attention")
    return made


def process_logits(logits: torch.Tensor, row_request: torch.Tensor | None = None,
                   history: torch.Tensor | None = None, history_offsets: torch.Tensor | None = None,
                   prompt_lens: torch.Tensor | None = None, repetition: torch.Tensor | None = None,
                   frequency: torch.Tensor | None = None, presence: torch.Tensor | None = None,
                   draft_tokens: torch.Tensor | None = None, cu_new: torch.Tensor | None = None,
                   tree_mask: torch.Tensor | None = None, bias_tokens: torch.Tensor | None = None,
                   bias_values: torch.Tensor | None = None, bias_offsets: torch.Tensor | None = None,
                   grammar_mask: torch.Tensor | None = None, grammar_rows: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """Repetition, frequency and presence penalties, biases and a grammar mask on
    logits [rows, vocab], in that order; ``out=logits`` works in place. Per-request
    tensors are indexed by ``row_request`` (the row itself if None); a drafted
    token's row counts the tokens of its path in ``tree_mask`` as generated."""
    made = (_step or _load()).process_logits(
        logits, row_request, history, history_offsets, prompt_lens, repetition, frequency, presence, draft_tokens, cu_new,
        tree_mask, bias_tokens, bias_values, bias_offsets, grammar_mask, grammar_rows, out)
    if type(made) is int:
        raise AWQError(made, "awq_process_logits")
    return made
