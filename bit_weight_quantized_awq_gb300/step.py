"""Torch-facing wrappers of the decoding step around the quantised layers:
allocate outputs, pass pointers, strides and the current stream to the C ABI
(``include/awq_gb300.h`` has the operators' definitions). No arithmetic happens
here, nothing waits for the GPU, and what is known on the device only (lengths,
table entries, tokens) is checked there: ``awq_last_device_status`` reports it.

A step is ``paged_plan`` -> per layer ``kv_append``, ``tree_attention`` ->
``process_logits``: the plan's ``cu_new``, ``slot_map`` and ``tree_mask`` are the
others' arguments.

A step's kernels take a few microseconds each, so the wrappers look at every
argument once, in one test; what is wrong is only looked for if that fails.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._binding import AWQError, DType, Status, awq_kv_append, awq_paged_plan, awq_process_logits, awq_tree_attention
from ._binding import pack_cache, pack_logits, pack_tree_attention
from .layer import _check, _stream

_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_DTYPES = {torch.float16: int(DType.F16), torch.bfloat16: int(DType.BF16), torch.float32: int(DType.F32)}
_CACHE_DTYPES = {torch.float16: int(DType.F16), torch.bfloat16: int(DType.BF16)}


class PagedPlan(NamedTuple):
    """What ``paged_plan`` lays out for a step (all on the device)."""
    cu_new: torch.Tensor          # int32 [B + 1]
    slot_map: torch.Tensor        # int64 [max_tokens]
    positions: torch.Tensor       # int32 [max_tokens]
    token_request: torch.Tensor   # int32 [max_tokens]
    tree_mask: torch.Tensor | None    # int32 [max_tokens, mask_words]
    counts: torch.Tensor          # int32 [2]: new tokens, blocks taken from free_blocks


def _cuda(t: torch.Tensor) -> torch.device:
    if not t.is_cuda:
        raise ValueError("the AWQ library runs on CUDA tensors only")
    return t.device


def _plain(t: torch.Tensor | None, dtype: torch.dtype, index: int) -> bool:
    """No tensor, or a contiguous one of `dtype` on device `index`."""
    return t is None or (t.dtype == dtype and t.get_device() == index and t.is_contiguous())


def _length(t: torch.Tensor | None, name: str, n: int):
    if t is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")


def _pointer(t: torch.Tensor | None, name: str, dtype: torch.dtype, dev: torch.device, index: int, n: int | None) -> int:
    """The data of a contiguous tensor of n elements (any number if None), 0 for none."""
    if t is None:
        return 0
    if t.dtype != dtype or t.get_device() != index or not t.is_contiguous() or (n is not None and t.numel() != n):
        _check(t, name, dtype, dev)
        if n is not None:
            _length(t, name, n)
    return t.data_ptr()


def _table(t: torch.Tensor, requests: int, index: int) -> int:
    """The table's row stride."""
    if t.dtype != _I32 or t.get_device() != index or t.dim() != 2:
        raise ValueError("block_table must be a torch.int32 [requests, blocks] tensor on the others' device")
    rows, width = t.shape
    stride, step = t.stride()
    if rows != requests or (step != 1 and width > 1):
        raise ValueError("block_table must be [requests, blocks] with adjacent entries in a row")
    return stride if rows > 1 else width


def paged_plan(context_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
               free_blocks: torch.Tensor, block_size: int, max_tokens: int,
               parents: torch.Tensor | None = None, mask_words: int = 0) -> PagedPlan:
    """One step's layout from request lengths: extends ``block_table`` in place
    with blocks from the start of ``free_blocks`` and gives every new token its
    cache slot, position and request, and with ``mask_words`` > 0 its ancestors in
    the drafted tree that ``parents`` describes (a chain if None)."""
    dev = _cuda(context_lens)
    at = dev.index
    B = context_lens.numel()
    if not (_plain(context_lens, _I32, at) and _plain(new_lens, _I32, at) and _plain(free_blocks, _I32, at)
            and _plain(parents, _I32, at) and new_lens.numel() == B):
        for t, name in ((context_lens, "context_lens"), (new_lens, "new_lens"), (free_blocks, "free_blocks"),
                        (parents, "parents")):
            if t is not None:
                _check(t, name, _I32, dev)
        _length(new_lens, "new_lens", B)
    if parents is not None:
        _length(parents, "parents", max_tokens)
    stride = _table(block_table, B, at)
    if max_tokens < 0 or mask_words < 0:
        raise ValueError("max_tokens and mask_words must not be negative")
    T = max_tokens
    cu_new = torch.empty(B + 1, dtype=_I32, device=dev)
    counts = torch.empty(2, dtype=_I32, device=dev)
    slot_map = torch.empty(T, dtype=_I64, device=dev)
    positions = torch.empty(T, dtype=_I32, device=dev)
    request = torch.empty(T, dtype=_I32, device=dev)
    tree_mask = torch.empty((T, mask_words), dtype=_I32, device=dev) if mask_words else None
    st = awq_paged_plan(context_lens.data_ptr(), new_lens.data_ptr(), B, block_table.data_ptr(), block_table.shape[1],
                        stride, free_blocks.data_ptr(), free_blocks.numel(), block_size,
                        None if parents is None else parents.data_ptr(), T, cu_new.data_ptr(), slot_map.data_ptr(),
                        positions.data_ptr(), request.data_ptr(), tree_mask.data_ptr() if mask_words else None,
                        mask_words, counts.data_ptr(), _stream(dev))
    if st != Status.OK:
        raise AWQError(st, "awq_paged_plan")
    return PagedPlan(cu_new, slot_map, positions, request, tree_mask, counts)


def _cache(t: torch.Tensor, name: str, dtype: torch.dtype, index: int, shape) -> tuple[int, int, int, int]:
    """(data, block, token and head stride) of a paged cache of this shape."""
    stride = t.stride()
    if t.dtype != dtype or t.get_device() != index or len(stride) != 4 or t.shape != shape or \
            (stride[3] != 1 and shape[3] > 1):
        raise ValueError(f"{name} must be a {dtype} [blocks, block_size, kv_heads, head_dim] tensor with adjacent "
                         f"head_dim elements on the others' device, of shape {tuple(shape)}")
    n, page, heads, dim = shape
    # the stride of an axis with one entry is never used: a valid one stands in
    return (t.data_ptr(), stride[0] if n > 1 else page * heads * dim, stride[1], stride[2] if heads > 1 else dim)


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, index: int):
    """(tokens, heads, head_dim, token stride, head stride)."""
    if t.dtype != dtype or t.get_device() != index:
        raise ValueError(f"{name} must be {dtype} on the others' device, got {t.dtype} on {t.device}")
    stride, shape = t.stride(), t.shape
    if len(stride) != 3 or (stride[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with adjacent head_dim elements")
    n, heads, dim = shape
    return n, heads, dim, stride[0] if n > 1 else heads * dim, stride[1] if heads > 1 else dim


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              slot_map: torch.Tensor) -> None:
    """Writes the new tokens' keys and values [tokens, kv_heads, head_dim] (views of
    a fused projection's output serve as they are) into the slots of a paged
    cache [blocks, block_size, kv_heads, head_dim]; slot -1 is skipped."""
    dev = _cuda(k_cache)
    at = dev.index
    dtype, shape = k_cache.dtype, k_cache.shape
    if dtype not in _CACHE_DTYPES:
        raise ValueError(f"the cache must be float16 or bfloat16, got {dtype}")
    kc, vc = _cache(k_cache, "k_cache", dtype, at, shape), _cache(v_cache, "v_cache", dtype, at, shape)
    T, heads, dim, kt, kh = _rows(k, "k", dtype, at)
    vT, v_heads, v_dim, vt, vh = _rows(v, "v", dtype, at)
    n, page, c_heads, c_dim = shape
    if not (T == vT and heads == v_heads == c_heads and dim == v_dim == c_dim):
        raise ValueError("k, v and the two caches must agree in heads and head_dim")
    if not _plain(slot_map, _I64, at) or slot_map.numel() != T:
        _check(slot_map, "slot_map", _I64, dev)
        _length(slot_map, "slot_map", T)
    st = awq_kv_append(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, pack_cache(*kc), pack_cache(*vc),
                       slot_map.data_ptr(), T, n, page, heads, dim, _stream(dev))
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
    at = dev.index
    dtype, shape = q.dtype, k_cache.shape
    if dtype not in _CACHE_DTYPES:
        raise ValueError(f"q must be float16 or bfloat16, got {dtype}")
    T, heads, dim, qt, qh = _rows(q, "q", dtype, at)
    kc, vc = _cache(k_cache, "k_cache", dtype, at, shape), _cache(v_cache, "v_cache", dtype, at, shape)
    n, page, kv_heads, kv_dim = shape
    if kv_dim != dim:
        raise ValueError("q and the caches must agree in head_dim")
    B = context_lens.numel()
    if not (_plain(context_lens, _I32, at) and _plain(cu_new, _I32, at) and cu_new.numel() == B + 1):
        _check(context_lens, "context_lens", _I32, dev)
        _check(cu_new, "cu_new", _I32, dev)
        _length(cu_new, "cu_new", B + 1)
    stride = _table(block_table, B, at)
    words = mask = 0
    if tree_mask is not None:
        if not _plain(tree_mask, _I32, at):
            _check(tree_mask, "tree_mask", _I32, dev)
        if tree_mask.dim() != 2 or tree_mask.shape[0] != T or tree_mask.shape[1] == 0:
            raise ValueError("tree_mask must be [tokens, mask_words]")
        words, mask = tree_mask.shape[1], tree_mask.data_ptr()
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _check(out, "out", dtype, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is not None:
        _check(lse, "lse", _F32, dev)
        if lse.shape != (T, heads):
            raise ValueError("lse must be [tokens, q_heads]")
    args = pack_tree_attention(q.data_ptr(), qt, qh, out.data_ptr(), 0 if lse is None else lse.data_ptr(), *kc, *vc,
                               block_table.data_ptr(), block_table.shape[1], stride, context_lens.data_ptr(),
                               cu_new.data_ptr(), mask, words, B, T, heads, kv_heads, dim, n, page, max_new,
                               max_context, scale, _CACHE_DTYPES[dtype])
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
    at = dev.index
    dtype = logits.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"logits must be float16, bfloat16 or float32, got {dtype}")
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [rows, vocab] with adjacent elements in a row")
    rows, vocab = logits.shape
    # the requests: the rows, or as many as the per-request tensors have
    if row_request is None:
        B = rows
    else:
        B = 2 ** 31 - 1      # if nothing is indexed by a request
        for t, more in ((repetition, 0), (frequency, 0), (presence, 0), (prompt_lens, 0), (history_offsets, 1),
                        (bias_offsets, 1), (cu_new, 1)):
            if t is not None:
                B = t.numel() - more
                break
    if bias_tokens is not None and (bias_values is None or bias_offsets is None):
        raise ValueError("bias_tokens, bias_values and bias_offsets go together")
    if history is not None and history_offsets is None:
        raise ValueError("history needs history_offsets")
    if draft_tokens is not None and cu_new is None:
        raise ValueError("draft_tokens needs cu_new")
    biases = None if bias_tokens is None else bias_tokens.numel()
    pointers = (
        _pointer(row_request, "row_request", _I32, dev, at, rows),
        _pointer(history, "history", _I32, dev, at, None),
        _pointer(history_offsets, "history_offsets", _I32, dev, at, B + 1),
        _pointer(prompt_lens, "prompt_lens", _I32, dev, at, B),
        0 if history is None else history.numel(),
        _pointer(repetition, "repetition", _F32, dev, at, B),
        _pointer(frequency, "frequency", _F32, dev, at, B),
        _pointer(presence, "presence", _F32, dev, at, B),
        _pointer(draft_tokens, "draft_tokens", _I32, dev, at, rows),
        _pointer(cu_new, "cu_new", _I32, dev, at, B + 1),
        _pointer(tree_mask, "tree_mask", _I32, dev, at, None))
    lists = (
        _pointer(bias_tokens, "bias_tokens", _I32, dev, at, None),
        _pointer(bias_offsets, "bias_offsets", _I32, dev, at, B + 1),
        _pointer(bias_values, "bias_values", _F32, dev, at, biases),
        biases or 0,
        _pointer(grammar_mask, "grammar_mask", _I32, dev, at, None),
        _pointer(grammar_rows, "grammar_rows", _I32, dev, at, rows))
    words = masks = 0
    if tree_mask is not None:
        if tree_mask.dim() != 2 or tree_mask.shape[0] != rows:
            raise ValueError("tree_mask must be [rows, mask_words]")
        words = tree_mask.shape[1]
    if grammar_mask is not None:
        if grammar_mask.dim() != 2 or grammar_mask.shape[1] != (vocab + 31) // 32:
            raise ValueError("grammar_mask must be [masks, ceil(vocab / 32)]")
        masks = grammar_mask.shape[0]
    if out is None:
        out = torch.empty_like(logits, memory_format=torch.contiguous_format)
    elif out is not logits:
        if out.dtype != dtype or out.device != dev or out.shape != logits.shape or \
                (out.stride(1) != 1 and vocab > 1):
            raise ValueError("out must be like logits, with adjacent elements in a row")
    args = pack_logits(logits.data_ptr(), out.data_ptr(), logits.stride(0) if rows > 1 else vocab,
                       out.stride(0) if rows > 1 else vocab, rows, vocab, B, *pointers, words, *lists, masks,
                       _DTYPES[dtype])
    st = awq_process_logits(args, _stream(dev))
    if st != Status.OK:
        raise AWQError(st, "awq_process_logits")
    return out
