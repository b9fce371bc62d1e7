"""Torch-facing functions of the decoding step around the quantised layers
(``include/awq_gb300.h`` has the operators' definitions). No arithmetic happens
here, nothing waits for the GPU, and what is known on the device only (lengths,
table entries, tokens) is checked there: ``awq_last_device_status`` reports it. The
tensors must be on the current CUDA device (``torch.cuda.set_device``), else ValueError.

A step is ``paged_plan`` -> per layer ``rotary_append`` (or ``rotary`` and ``kv_append``),
``tree_attention`` -> ``process_logits``: the plan's ``positions``, ``cu_new``, ``slot_map``
and ``tree_mask`` are the others' arguments. With beams, ``beam_select`` -> ``reorder_states``,
``fork_pages``, ``copy_pages`` -> ``free_pages`` come after it, whose list of free blocks the
next plan takes from: nothing of this waits for the host.

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
                  (lib.awq_paged_plan, lib.awq_kv_append, lib.awq_tree_attention, lib.awq_process_logits,
                   lib.awq_rotary, lib.awq_beam_select, lib.awq_beam_select_workspace, lib.awq_reorder_states,
                   lib.awq_fork_pages, lib.awq_copy_pages, lib.awq_free_pages, lib.awq_compact_pages,
                   lib.awq_pages_workspace)))
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
    the drafted tree that ``parents`` describes (a chain if None). ``free_blocks`` may
    be ``free_pages``' whole list: an entry of -1 means that none is left (slots of -1,
    ERR_TOO_LARGE in the device status)."""
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


def rotary_axes(sections: list[int], interleaved: bool = False, device="cuda") -> torch.Tensor:
    """The ``axes`` of ``rotary`` for frequencies shared out among axes (time, height, width, say):
    ``sections[a]`` of them belong to axis a, in blocks one after the other, or
    ``interleaved``: dealt out in turn for as long as an axis has some left."""
    if not sections or any(n < 0 for n in sections):
        raise ValueError("sections must be numbers of frequencies, one for each axis")
    if interleaved:
        order = [a for i in range(max(sections)) for a, n in enumerate(sections) if i < n]
    else:
        order = [a for a, n in enumerate(sections) for _ in range(n)]
    return torch.tensor(order, dtype=torch.int32, device=device)


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
           axes: torch.Tensor | None = None, pairs: bool = False, q_out: torch.Tensor | None = None,
           k_out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """q and k [tokens, heads, head_dim] turned by their tokens' ``positions`` (int32
    [tokens], the plan's, or [axes, tokens] with ``axes`` saying which one each
    frequency goes by). ``inv_freq`` (fp32) has half as many entries as elements of a head
    are turned; element i is paired with the one half of them further, or with its neighbour
    (``pairs``). Views of a fused projection's output serve as they are; ``q_out=q`` and
    ``k_out=k`` work in place."""
    made = (_step or _load()).rotary(q, k, positions, inv_freq, axes, pairs, q_out, k_out)
    if type(made) is int:
        raise AWQError(made, "awq_rotary")
    return made


def rotary_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, slot_map: torch.Tensor,
                  axes: torch.Tensor | None = None, pairs: bool = False,
                  q_out: torch.Tensor | None = None) -> torch.Tensor:
    """``rotary`` and ``kv_append`` in one pass: returns the turned q; the turned keys and the
    values go into their slots of the paged cache."""
    made = (_step or _load()).rotary_append(q, k, v, positions, inv_freq, k_cache, v_cache, slot_map, axes, pairs, q_out)
    if type(made) is int:
        raise AWQError(made, "awq_rotary")
    return made


class BeamStep(NamedTuple):
    """What ``beam_select`` keeps (all on the device): -inf, -1, -1 where there are fewer."""
    scores: torch.Tensor          # fp32 [requests, num_beams], in descending order
    parents: torch.Tensor         # int32 [requests, num_beams]: rows of the logits
    tokens: torch.Tensor          # int32 [requests, num_beams]
    ended_scores: torch.Tensor | None     # the same of the candidates that end; None without end_tokens
    ended_parents: torch.Tensor | None
    ended_tokens: torch.Tensor | None


def beam_select(logits: torch.Tensor, scores: torch.Tensor, num_beams: int,
                end_tokens: torch.Tensor | None = None) -> BeamStep:
    """The best continuations of every request's beams: ``scores`` (fp32 [requests, beams],
    -inf for a beam that is none) plus the log-softmax of their logits [requests * beams, vocab]. The
    first ``num_beams`` whose token is not one of ``end_tokens`` go on; those among the first
    ``num_beams`` of all that end are given apart. Equal scores: the lower row, then the lower token."""
    made = (_step or _load()).beam_select(logits, scores, num_beams, end_tokens)
    if type(made) is int:
        raise AWQError(made, "awq_beam_select")
    return BeamStep._make(made)


def reorder_states(states: list[torch.Tensor], parents: torch.Tensor,
                   outs: list[torch.Tensor] | None = None) -> list[torch.Tensor]:
    """Rows ``parents`` (int32 [rows]) of every tensor of ``states`` [rows, ...], whatever its type:
    token histories, recurrent states. -1 gives zeros. ``outs`` must not overlap ``states``."""
    made = (_step or _load()).reorder_states(states, parents, outs)
    if type(made) is int:
        raise AWQError(made, "awq_reorder_states")
    return made


class ForkedPages(NamedTuple):
    """What ``fork_pages`` lays out (all on the device, in one allocation)."""
    block_table: torch.Tensor     # int32 [rows, width]
    lens: torch.Tensor            # int32 [rows]
    src: torch.Tensor             # int32 [rows]: what copy_pages has to copy, -1 after the last
    dst: torch.Tensor
    tokens: torch.Tensor
    count: torch.Tensor           # int32 [1]: how many that are, as many blocks were taken


def fork_pages(block_table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor, free_blocks: torch.Tensor,
               block_size: int, free_start: torch.Tensor | None = None) -> ForkedPages:
    """Block tables of the rows that go on from rows ``parents`` (``beam_select``'s, flat) of
    ``block_table``, which hold ``lens`` tokens. Full pages are shared; a partly filled last one
    stays with its first child, the others take blocks from ``free_blocks`` (from
    ``free_start`` on: a plan's ``counts[1:]``, say) and a copy, which
    ``copy_pages(caches, f.src, f.dst, f.tokens, f.count)`` makes. Where no block is left (the
    list's end, or an entry of -1), the row's last page is -1 and the device status ERR_TOO_LARGE."""
    made = (_step or _load()).fork_pages(block_table, lens, parents, free_blocks, block_size, free_start)
    if type(made) is int:
        raise AWQError(made, "awq_fork_pages")
    return ForkedPages._make(made)


def copy_pages(caches: list[torch.Tensor], src: torch.Tensor, dst: torch.Tensor, tokens: torch.Tensor | None = None,
               count: torch.Tensor | None = None) -> None:
    """Blocks ``src`` to blocks ``dst`` within every cache of a list (the keys and values of all
    layers, of one shape), only their first ``tokens``, and only the first ``count`` (int32
    [1]) of the pairs if given. All at once: no dst is another pair's src or dst."""
    status = (_step or _load()).copy_pages(caches, src, dst, tokens, count)
    if status is not None:
        raise AWQError(status, "awq_copy_pages")


class FreePages(NamedTuple):
    """What ``free_pages`` finds (all on the device)."""
    free_blocks: torch.Tensor     # int32 [num_blocks]: ascending, -1 after the last
    counts: torch.Tensor          # int32 [2]: free blocks, used blocks


def free_pages(block_table: torch.Tensor, lens: torch.Tensor, block_size: int, num_blocks: int,
               held: torch.Tensor | None = None) -> FreePages:
    """The blocks of a cache that none of the rows needs for its ``lens`` tokens and that are
    not among ``held`` (int32; -1 is skipped): the free list of the next plan or fork. To
    free a request, set its length to 0."""
    made = (_step or _load()).free_pages(block_table, lens, block_size, num_blocks, held)
    if type(made) is int:
        raise AWQError(made, "awq_free_pages")
    return FreePages._make(made)


class CompactPages(NamedTuple):
    """What ``compact_pages`` lays out (all on the device, in one allocation)."""
    block_table: torch.Tensor     # int32 [rows, width], with the new numbers
    block_map: torch.Tensor       # int32 [num_blocks]: a block's new number, -1 for a free one
    src: torch.Tensor             # int32 [num_blocks // 2]: what copy_pages has to copy, -1 after the last
    dst: torch.Tensor
    count: torch.Tensor           # int32 [1]: how many that are


def compact_pages(block_table: torch.Tensor, lens: torch.Tensor, block_size: int, num_blocks: int,
                  held: torch.Tensor | None = None) -> CompactPages:
    """Moves the used blocks (as in ``free_pages``) to the cache's beginning: those that lie past
    it take the free blocks there. ``copy_pages(caches, c.src, c.dst, count=c.count)`` moves
    their contents, ``block_map`` renames a caller's own ``held``."""
    made = (_step or _load()).compact_pages(block_table, lens, block_size, num_blocks, held)
    if type(made) is int:
        raise AWQError(made, "awq_compact_pages")
    return CompactPages._make(made)
