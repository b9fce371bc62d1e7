"""The decoding step's operators in 64 bits, request by request and token by
token, on the CPU: what the GPU tests compare with."""
from __future__ import annotations

import numpy as np
import torch


def plan(ctx, new, table, free, page, parents=None, words=0):
    """(cu_new, table, slots, positions, request, mask [tokens, words] uint32, counts)."""
    table = table.copy()
    cu, taken = [0], 0
    slots, positions, request, masks = [], [], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        have, need = -(-c // page), -(-(c + n) // page)
        for j in range(have, need):
            table[b, j] = free[taken]
            taken += 1
        rows = []
        for i in range(n):
            up = i - 1 if parents is None else int(parents[cu[-1] + i])
            own = {i} | (rows[up] if up >= 0 else set())
            rows.append(own)
            slots.append(int(table[b, (c + i) // page]) * page + (c + i) % page)
            positions.append(c + len(own) - 1)
            request.append(b)
            m = np.zeros(words, dtype=np.uint32)
            for j in own:
                if j < 32 * words:
                    m[j // 32] |= np.uint32(1 << (j % 32))
            masks.append(m)
        cu.append(cu[-1] + n)
    return cu, table, slots, positions, request, np.array(masks, dtype=np.uint32).reshape(len(masks), words), [cu[-1], taken]


def attention(q, k_cache, v_cache, table, ctx, cu, scale, mask=None):
    """(out, lse, sum of weight * |v|) in float64. A key that a row does not see
    takes no part in its row, whatever it holds. mask: bool [tokens, max drafted]."""
    q, k_cache, v_cache = (t.detach().cpu().double() for t in (q, k_cache, v_cache))
    T, H, D = q.shape
    page, K = k_cache.shape[1:3]
    G = H // K
    out, lse = torch.zeros(T, H, D, dtype=torch.float64), torch.full((T, H), -torch.inf, dtype=torch.float64)
    size = torch.zeros(T, H, D, dtype=torch.float64)
    for b in range(len(ctx)):
        keys = ctx[b] + cu[b + 1] - cu[b]
        blocks = torch.as_tensor(table[b][:-(-keys // page)]).long()
        k = k_cache[blocks].flatten(0, 1)[:keys]
        v = v_cache[blocks].flatten(0, 1)[:keys]
        for t in range(cu[b], cu[b + 1]):
            n = cu[b + 1] - cu[b]
            drafted = torch.zeros(n, dtype=torch.bool)
            if mask is None:
                drafted[:t - cu[b] + 1] = True
            else:
                w = min(n, mask.shape[1])
                drafted[:w] = torch.as_tensor(mask[t][:w])
            at = torch.cat([torch.arange(ctx[b]), ctx[b] + drafted.nonzero()[:, 0]])
            if len(at) == 0:
                continue
            for h in range(H):
                s = (k[at, h // G] @ q[t, h]) * scale
                lse[t, h] = torch.logsumexp(s, 0)
                w = torch.softmax(s, 0)
                out[t, h] = w @ v[at, h // G]
                size[t, h] = w @ v[at, h // G].abs()
    return out, lse, size


def logits(x, req, B, hist=None, prompt=None, rep=None, freq=None, pres=None, path=None, bias=None, allowed=None):
    """float64 [rows, vocab]. hist: list of token lists; path: list of token lists
    a row; bias: list of [(token, value)]; allowed: bool [rows, vocab]."""
    x = x.detach().cpu().double().numpy().copy()
    V = x.shape[1]
    for r in range(x.shape[0]):
        b = int(req[r])
        h = np.asarray([] if hist is None else hist[b], dtype=np.int64)
        cut = 0 if prompt is None else prompt[b]
        mine = np.asarray([] if path is None else path[r], dtype=np.int64)
        said = np.concatenate([h[cut:], mine])
        known = np.unique(np.concatenate([h, mine]))
        known, said = known[known >= 0].astype(np.int64), said[said >= 0].astype(np.int64)
        if rep is not None:
            x[r, known] = np.where(x[r, known] > 0, x[r, known] / rep[b], x[r, known] * rep[b])
        count = np.bincount(said, minlength=V)
        seen = count > 0
        x[r, seen] -= (0 if freq is None else freq[b]) * count[seen] + (0 if pres is None else pres[b])
        for token, value in ([] if bias is None else bias[b]):
            x[r, token] += value
        if allowed is not None:
            x[r, ~allowed[r]] = -np.inf
    return x
