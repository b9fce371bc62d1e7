"""Rotary positions, beam search and the calls on a cache's pages in 64 bits or more, item by
item, on the CPU: what the GPU tests compare with."""
from __future__ import annotations

import numpy as np


def rotary(x, positions, inv_freq, axes=None, pairs=False):
    """(turned x, sum of the two products' sizes), float64 [tokens, heads, dim]; the angles in extended precision.
    positions: int [axes, tokens]."""
    x = np.asarray(x, dtype=np.float64)
    n = len(inv_freq)
    axes = np.zeros(n, dtype=int) if axes is None else np.asarray(axes)
    angle = np.asarray(positions, dtype=np.longdouble)[axes].T * np.asarray(inv_freq, dtype=np.longdouble)
    cos, sin = np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if pairs else (slice(0, n), slice(n, 2 * n))
    u, w = x[..., first], x[..., second]
    out, size = x.copy(), np.zeros_like(x)
    out[..., first], out[..., second] = u * cos - w * sin, w * cos + u * sin
    size[..., first] = size[..., second] = np.abs(u) + np.abs(w)
    return out, size


def scores(logits, before):
    """float64 [requests, beams, vocab] of all candidates, -inf where there is none."""
    B, W = before.shape
    x = np.asarray(logits, dtype=np.float64).reshape(B, W, -1)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        top = x.max(-1, keepdims=True)
        total = np.log(np.exp(x - top).sum(-1, keepdims=True))
        # not x - (top + total): next to a top of -3.4e38 the total would be lost, since 64 bits have steps of 2^75 there
        s = np.asarray(before, dtype=np.float64)[..., None] + ((x - top) - total)
    sound = np.isfinite(top) & np.isfinite(total) & np.isfinite(before)[..., None]
    return np.where(sound & (x > -np.inf), s, -np.inf)


def beams(logits, before, keep, ends=()):
    """(live, ended): for each request a list of (score, row, token), in order."""
    every = scores(logits, before)
    B, W, V = every.shape
    live, ended = [], []
    for b in range(B):
        flat = every[b].reshape(-1)
        x = np.asarray(logits, dtype=np.float64)[b * W:(b + 1) * W].reshape(-1) + 0.0
        row, token = np.divmod(np.arange(W * V), V)
        best = np.lexsort((token, -np.where(flat > -np.inf, x, 0), row, -flat))
        mine, gone = [], []
        for rank, i in enumerate(best):
            if flat[i] == -np.inf or len(mine) == keep:
                break
            item = (flat[i], b * W + int(row[i]), int(token[i]))
            if item[2] in ends:
                if rank < keep:
                    gone.append(item)
            else:
                mine.append(item)
        live.append(mine)
        ended.append(gone)
    return live, ended


def fork(table, lens, parents, free, page, start=0):
    """(table, lens, [(src, dst, tokens)])."""
    new = np.full((len(parents), table.shape[1]), -1, dtype=np.int64)
    new_lens, pairs, seen = [], [], set()
    for r, p in enumerate(parents):
        n = lens[p] if p >= 0 else 0
        new_lens.append(n)
        have = -(-n // page)
        if p >= 0:
            new[r, :have] = table[p, :have]
        if n % page and p in seen:
            to = free[start + len(pairs)]
            pairs.append((int(table[p, have - 1]), int(to), n % page))
            new[r, have - 1] = to
        seen.add(p)
    return new, new_lens, pairs


def used(table, lens, page, blocks, held=()):
    """Truth values [blocks]."""
    got = np.zeros(blocks, dtype=bool)
    for row, n in zip(table, lens):
        got[row[:-(-n // page)]] = True
    for b in held:
        if b >= 0:
            got[b] = True
    return got


def compact(table, lens, page, blocks, held=()):
    """(table, map, [(src, dst)])."""
    u = used(table, lens, page, blocks, held)
    n = int(u.sum())
    moving, holes = [b for b in range(n, blocks) if u[b]], [b for b in range(n) if not u[b]]
    to = np.where(u, np.arange(blocks), -1)
    to[moving] = holes
    new = np.full(table.shape, -1, dtype=np.int64)
    for r, (row, length) in enumerate(zip(table, lens)):
        have = -(-length // page)
        new[r, :have] = to[row[:have]]
    return new, to, list(zip(moving, holes))
