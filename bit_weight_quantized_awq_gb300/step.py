"""Torch-facing wrappers of the decoding step around the quantised layers:
allocate outputs, pass pointers, strides and the current stream to the C ABI
(``include/awq_gb300.h`` has the operators' definitions). No arithmetic happens
here, nothing waits for the GPU, and what is known on the device only (lengths,
table entries, tokens) is checked there: ``awq_last_device_status`` reports it.

A step is ``paged_plan`` -> per layer ``kv_append``, ``tree_attention`` ->
``process_logits``: the plan's ``cu_new``, ``slot_map`` and ``tree_mask`` are the
others' arguments.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._binding import (AWQError, Cache, DType, Logits, Status, TreeAttention, awq_kv_append, awq_paged_plan,
                       awq_process_logits, awq_tree_attention)
from .layer import _check, _ptr, _stream

_I32 = torch.int32
_DTYPES = {torch.float16: DType.F16, torch.bfloat16: DType.BF16, torch.float32: DType.F32}


class PagedPlan(NamedTuple):
    """What ``paged_plan`` lays out for a step (all on the device)."""
    cu_new: torch.Tensor          # int32 [B + 1]
    slot_map: torch.Tensor        # int64 [max_tokens]
    positions: torch.Tensor       # int32 [max_tokens]
    token_request: torch.Tensor   # int32 [max_tokens]
    tree_mask: torch.Tensor | None    # int32 [max_tokens, mask_words]
    counts: torch.Tensor          # int32 [2]: new tokens, blocks taken from free_blocks


def _cuda(t: torch.Tensor) -> torch.device:
    dev = t.device
    if dev.type != "cuda":
        raise ValueError("the AWQ library runs on CUDA tensors only")
    return dev


def _ints(dev: torch.device, **tensors):
    """Every given tensor is a contiguous int32 tensor on `dev`."""
    for name, t in tensors.items():
        if t is not None and not (t.dtype == _I32 and t.device == dev and t.is_contiguous()):
            _check(t, name, _I32, dev)


def _length(t: torch.Tensor | None, name: str, n: int):
    if t is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")


def _table(block_table: torch.Tensor, requests: int, dev: torch.device):
    if block_table.dtype != _I32 or block_table.device != dev:
        raise ValueError(f"block_table must be torch.int32 on {dev}")
    if block_table.dim() != 2 or block_table.shape[0] != requests or block_table.stride(1) != 1:
        raise ValueError("block_table must be [requests, blocks] with adjacent entries in a row")


def paged_plan(context_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
               free_blocks: torch.Tensor, block_size: int, max_tokens: int,
               parents: torch.Tensor | None = None, mask_words: int = 0) -> PagedPlan:
    """One step's layout from request lengths: extends ``block_table`` in place
    with blocks from the start of ``free_blocks`` and gives every new token its
    cache slot, position and request, and with ``mask_words`` > 0 its ancestors in
    the drafted tree that ``parents`` describes (a chain if None)."""
    dev = _cuda(context_lens)
    B = context_lens.numel()
    _ints(dev, context_lens=context_lens, new_lens=new_lens, free_blocks=free_blocks, parents=parents)
    _length(new_lens, "new_lens", B)
    _length(parents, "parents", max_tokens)
    _table(block_table, B, dev)
    if max_tokens < 0 or mask_words < 0:
        raise ValueError("max_tokens and mask_words must not be negative")
    cu_new = torch.empty(B + 1, dtype=_I32, device=dev)
    counts = torch.empty(2, dtype=_I32, device=dev)
    slot_map = torch.empty(max_tokens, dtype=torch.int64, device=dev)
    positions = torch.empty(max_tokens, dtype=_I32, device=dev)
    token_request = torch.empty(max_tokens, dtype=_I32, device=dev)
    tree_mask = torch.empty((max_tokens, mask_words), dtype=_I32, device=dev) if mask_words else None
    st = awq_paged_plan(context_lens.data_ptr(), new_lens.data_ptr(), B, block_table.data_ptr(), block_table.shape[1],
                        block_table.stride(0) if B > 1 else block_table.shape[1], free_blocks.data_ptr(),
                        free_blocks.numel(), block_size, _ptr(parents), max_tokens, cu_new.data_ptr(),
                        slot_map.data_ptr(), positions.data_ptr(), token_request.data_ptr(), _ptr(tree_mask),
                        mask_words, counts.data_ptr(), _stream(dev))
    if st != Status.OK:
        raise AWQError(st, "awq_paged_plan")
    return PagedPlan(cu_new, slot_map, positions, token_request, tree_mask, counts)


def _cache(t: torch.Tensor, name: str, dtype: torch.dtype, dev: torch.device) -> Cache:
    if t.dtype != dtype or t.device != dev:
        raise ValueError(f"{name} must be {dtype} on {dev}, got {t.dtype} on {t.device}")
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be [blocks, block_size, kv_heads, head_dim] with adjacent head_dim elements")
    n, page, heads, dim = t.shape
    s = t.stride()
    # the stride of an axis with one entry is never used: a valid one stands in
    return Cache(t.data_ptr(), s[0] if n > 1 else page * heads * dim, s[1], s[2] if heads > 1 else dim)


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, dev: torch.device):
    """(token stride, head stride) of [tokens, heads, head_dim]."""
    if t.dtype != dtype or t.device != dev:
        raise ValueError(f"{name} must be {dtype} on {dev}, got {t.dtype} on {t.device}")
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with adjacent head_dim elements")
    n, heads, dim = t.shape
    s = t.stride()
    return s[0] if n > 1 else heads * dim, s[1] if heads > 1 else dim


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              slot_map: torch.Tensor) -> None:
    """Writes the new tokens' keys and values [tokens, kv_heads, head_dim] (views of
    a fused projection's output serve as they are) into the slots of a paged
    cache [blocks, block_size, kv_heads, head_dim]; slot -1 is skipped."""
    dev = _cuda(k_cache)
    dtype = k_cache.dtype
    if dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"the cache must be float16 or bfloat16, got {dtype}")
    kc, vc = _cache(k_cache, "k_cache", dtype, dev), _cache(v_cache, "v_cache", dtype, dev)
    (kt, kh), (vt, vh) = _rows(k, "k", dtype, dev), _rows(v, "v", dtype, dev)
    n, page, heads, dim = k_cache.shape
    if v_cache.shape != k_cache.shape or k.shape != v.shape or k.shape[1:] != (heads, dim):
        raise ValueError("k, v and the two caches must agree in heads and head_dim")
    _check(slot_map, "slot_map", torch.int64, dev)
    _length(slot_map, "slot_map", k.shape[0])
    st = awq_kv_append(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, kc, vc, slot_map.data_ptr(), k.shape[0], n, page,
                       heads, dim, _stream(dev))
    if st != Status.OK:
        raise AWQError(st, "awq_kv_append")


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                   context_lens: torch.Tensor, cu_new: torch.Tensor, scale: float, max_new: int, max_context: int,
                   tree_mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None) -> torch.Tensor:
    """softmax(scale q k^T) v of new tokens [tokens, q_heads, head_dim] over their
    requests' caches, their own keys and values included: a token sees its whole
    context and, of the new tokens, those of its ``tree_mask`` row (itself and
    the ones before it if None). ``max_new`` and ``max_context`` bound the
    lengths; ``lse`` (fp32 [tokens, q_heads]) receives the log-sum-exp."""
    dev = _cuda(q)
    dtype = q.dtype
    if dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"q must be float16 or bfloat16, got {dtype}")
    qt, qh = _rows(q, "q", dtype, dev)
    kc, vc = _cache(k_cache, "k_cache", dtype, dev), _cache(v_cache, "v_cache", dtype, dev)
    tokens, heads, dim = q.shape
    n, page, kv_heads, kv_dim = k_cache.shape
    if v_cache.shape != k_cache.shape or kv_dim != dim:
        raise ValueError("q and the two caches must agree in head_dim, the caches in every size")
    B = context_lens.numel()
    _ints(dev, context_lens=context_lens, cu_new=cu_new, tree_mask=tree_mask)
    _length(cu_new, "cu_new", B + 1)
    _table(block_table, B, dev)
    words = 0
    if tree_mask is not None:
        if tree_mask.dim() != 2 or tree_mask.shape[0] != tokens:
            raise ValueError("tree_mask must be [tokens, mask_words]")
        words = tree_mask.shape[1]
        if words == 0:
            raise ValueError("tree_mask has no words")
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=dtype, device=dev)
    else:
        _check(out, "out", dtype, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is not None:
        _check(lse, "lse", torch.float32, dev)
        if lse.shape != (tokens, heads):
            raise ValueError("lse must be [tokens, q_heads]")
    args = TreeAttention(q.data_ptr(), qt, qh, out.data_ptr(), _ptr(lse), kc, vc, block_table.data_ptr(),
                         block_table.shape[1], block_table.stride(0) if B > 1 else block_table.shape[1],
                         context_lens.data_ptr(), cu_new.data_ptr(), _ptr(tree_mask), words, B, tokens, heads,
                         kv_heads, dim, n, page, max_new, max_context, scale, _DTYPES[dtype])
    st = awq_tree_attention(args, _stream(dev))
    if st != Status.OK:
        raise AWQError(st, "awq_tree_attention")
    return out


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
    dev = _cuda(logits)
    dtype = logits.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"logits must be float16, bfloat16 or float32, got {dtype}")
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [rows, vocab] with adjacent elements in a row")
    rows, vocab = logits.shape
    # the requests: the rows, or as many as the per-request tensors have
    B = rows if row_request is None else None
    for t, name, more in ((repetition, "repetition", 0), (frequency, "frequency", 0), (presence, "presence", 0),
                          (prompt_lens, "prompt_lens", 0), (history_offsets, "history_offsets", 1),
                          (bias_offsets, "bias_offsets", 1), (cu_new, "cu_new", 1)):
        if t is None:
            continue
        if B is None:
            B = t.numel() - more
        _length(t, name, B + more)
    if B is None:
        B = 2 ** 31 - 1      # nothing is indexed by a request
    for t, name in ((repetition, "repetition"), (frequency, "frequency"), (presence, "presence"),
                    (bias_values, "bias_values")):
        if t is not None and not (t.dtype == torch.float32 and t.device == dev and t.is_contiguous()):
            _check(t, name, torch.float32, dev)
    _ints(dev, row_request=row_request, history=history, history_offsets=history_offsets, prompt_lens=prompt_lens,
          draft_tokens=draft_tokens, cu_new=cu_new, tree_mask=tree_mask, bias_tokens=bias_tokens,
          bias_offsets=bias_offsets, grammar_mask=grammar_mask, grammar_rows=grammar_rows)
    _length(row_request, "row_request", rows)
    _length(draft_tokens, "draft_tokens", rows)
    _length(grammar_rows, "grammar_rows", rows)
    if bias_tokens is not None:
        if bias_values is None or bias_offsets is None:
            raise ValueError("bias_tokens, bias_values and bias_offsets go together")
        _length(bias_values, "bias_values", bias_tokens.numel())
    if history is not None and history_offsets is None:
        raise ValueError("history needs history_offsets")
    if draft_tokens is not None and cu_new is None:
        raise ValueError("draft_tokens needs cu_new")
    if tree_mask is not None and (tree_mask.dim() != 2 or tree_mask.shape[0] != rows):
        raise ValueError("tree_mask must be [rows, mask_words]")
    if grammar_mask is not None and (grammar_mask.dim() != 2 or grammar_mask.shape[1] != (vocab + 31) // 32):
        raise ValueError("grammar_mask must be [masks, ceil(vocab / 32)]")
    if out is None:
        out = torch.empty((rows, vocab), dtype=dtype, device=dev)
    elif out is not logits:
        if out.dtype != dtype or out.device != dev or out.shape != logits.shape or \
                (out.stride(1) != 1 and vocab > 1):
            raise ValueError("out must be like logits, with adjacent elements in a row")
    args = Logits(logits.data_ptr(), out.data_ptr(), logits.stride(0) if rows > 1 else vocab,
                  out.stride(0) if rows > 1 else vocab, rows, vocab, B, _ptr(row_request), _ptr(history),
                  _ptr(history_offsets), _ptr(prompt_lens), 0 if history is None else history.numel(),
                  _ptr(repetition), _ptr(frequency), _ptr(presence), _ptr(draft_tokens), _ptr(cu_new),
                  _ptr(tree_mask), 0 if tree_mask is None else tree_mask.shape[1], _ptr(bias_tokens),
                  _ptr(bias_offsets), _ptr(bias_values), 0 if bias_tokens is None else bias_tokens.numel(),
                  _ptr(grammar_mask), _ptr(grammar_rows), 0 if grammar_mask is None else grammar_mask.shape[0],
                  _DTYPES[dtype])
    st = awq_process_logits(args, _stream(dev))
    if st != Status.OK:
        raise AWQError(st, "awq_process_logits")
    return out
