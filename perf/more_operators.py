"""Measured cases of the decoding step's rotary positions, beam search and cache
pages: ``rotary`` and ``rotary_append``, ``beam_select`` with ``reorder_states``,
``fork_pages`` and ``compact_pages`` with ``copy_pages``, ``free_pages``.

``run`` computes a case with the package's operators where ``own`` is true and
with elementary torch operations where it is false; ``exact`` computes what is
arithmetic in them from the definitions in 64 bits. What a case costs (lengths,
how many pages are copied) is a function of the case alone: a seed changes values,
orders and places.
"""
import random

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token of one request, 32 heads (a 4096-wide layer), into the cache: latency
        {"name": "rotary_one", "op": "rotary", "tokens": 1, "heads": 32, "kv_heads": 32, "dim": 128, "rotated": 128,
         "axes": 1, "cycle": False, "pairs": False, "append": True, "page": 16, "far": 8000, "dtype": "fp16"},
        # prompts being filled in, grouped heads (an 8192-wide layer's 64 / 8), into the cache, far positions
        {"name": "rotary_prompt", "op": "rotary", "tokens": 16383, "heads": 64, "kv_heads": 8, "dim": 128,
         "rotated": 128, "axes": 1, "cycle": False, "pairs": False, "append": True, "page": 64, "far": 1000000,
         "dtype": "bf16"},
        # a video's patches, time, height and width, few heads, not into a cache
        {"name": "rotary_video", "op": "rotary", "tokens": 30001, "heads": 16, "kv_heads": 4, "dim": 96, "rotated": 96,
         "axes": 3, "cycle": True, "pairs": False, "append": False, "page": 16, "far": 20000, "dtype": "bf16"},
        # four beams of one request: latency
        {"name": "beam_one", "op": "beam", "requests": 1, "beams": 4, "keep": 4, "vocab": 32000, "ends": 1,
         "history": 700, "masked": False, "dtype": "fp16"},
        # a serving batch, a large vocabulary
        {"name": "beam_b64", "op": "beam", "requests": 64, "beams": 8, "keep": 8, "vocab": 131072, "ends": 2,
         "history": 2000, "masked": False, "dtype": "bf16"},
        # wide beams over fp32 logits that a grammar mask has gone over
        {"name": "beam_wide", "op": "beam", "requests": 15, "beams": 32, "keep": 32, "vocab": 100003, "ends": 3,
         "history": 500, "masked": True, "dtype": "fp32"},
        # the pages of four beams of two requests, a small model
        {"name": "fork_small", "op": "fork", "requests": 2, "beams": 4, "context": 500, "page": 16, "layers": 2,
         "kv_heads": 8, "dim": 64, "dtype": "fp16"},
        # a serving batch: 24 layers' keys and values
        {"name": "fork_b48", "op": "fork", "requests": 48, "beams": 8, "context": 420, "page": 64, "layers": 24,
         "kv_heads": 8, "dim": 128, "dtype": "bf16"},
        # a decode batch's pages in a cache of a few hundred thousand tokens
        {"name": "free_b256", "op": "free", "rows": 256, "context": 4096, "page": 16, "spare": 0.3},
        # thousands of beams over a cache of millions of tokens
        {"name": "free_b4000", "op": "free", "rows": 4000, "context": 16384, "page": 16, "spare": 0.1},
        # a small cache, a few pages out of place
        {"name": "compact_small", "op": "compact", "rows": 12, "context": 700, "page": 16, "layers": 1, "kv_heads": 4,
         "dim": 128, "moved": 0.1, "spare": 0.5, "dtype": "fp16"},
        # a cache after a batch has ended: a third of the pages move down
        {"name": "compact_b64", "op": "compact", "rows": 64, "context": 2048, "page": 32, "layers": 8, "kv_heads": 8,
         "dim": 128, "moved": 0.33, "spare": 1.0, "dtype": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm, odd when above 64."""
    v = int(round(low * (high / low) ** rng.random()))
    return v if v <= 64 else min(high, v) - (1 - min(high, v) % 2)


def draw(rng):
    op = rng.choice(["rotary", "rotary", "beam", "beam", "fork", "free", "compact"])
    if op == "rotary":
        kv_heads, group = rng.choice([(32, 1), (8, 4), (8, 8), (4, 7), (1, 16), (2, 5)])
        dim, rotated = rng.choice([(64, 64), (64, 32), (80, 80), (80, 32), (96, 96), (128, 128), (128, 64), (256, 256),
                                   (72, 36)])
        axes = rng.choice([1, 1, 3])
        case = {"op": op, "tokens": _spread(rng, 1, 32767), "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
                "rotated": rotated, "axes": axes, "cycle": axes > 1 and rng.random() < 0.5,
                "pairs": rng.random() < 0.3, "append": rng.random() < 0.6, "page": rng.choice([16, 32, 64, 128]),
                "far": _spread(rng, 100, 4000001), "dtype": rng.choice(["fp16", "bf16"])}
        while work(case)["bytes"] > 6.5e8:
            case["tokens"] = case["tokens"] // 2
        return case
    if op == "beam":
        keep = rng.choice([1, 2, 4, 5, 8, 16, 32])
        case = {"op": op, "requests": _spread(rng, 1, 128), "beams": rng.choice([keep, keep, keep, 1, 7]), "keep": keep,
                "vocab": _spread(rng, 20000, 160001), "ends": rng.choice([0, 1, 3, 8]), "history": _spread(rng, 1, 4095),
                "masked": rng.random() < 0.4, "dtype": rng.choice(["fp16", "bf16", "fp32"])}
        while work(case)["bytes"] > 1.4e8:
            case["requests"] = (case["requests"] + 1) // 2
            if case["requests"] == 1:
                case["vocab"] = case["vocab"] // 4 * 2 + 1
        return case
    if op == "fork":
        case = {"op": op, "requests": _spread(rng, 1, 128), "beams": rng.choice([2, 3, 4, 8, 16]),
                "context": _spread(rng, 1, 4095), "page": rng.choice([16, 32, 64, 128]), "layers": _spread(rng, 1, 40),
                "kv_heads": rng.choice([1, 2, 8, 16]), "dim": rng.choice([64, 80, 128]),
                "dtype": rng.choice(["fp16", "bf16"])}
        while _cache_bytes(case, sum(_fork_pages(case)[1])) > 5e9 or work(case)["bytes"] > 1e9:
            case["requests"] = (case["requests"] + 1) // 2
            case["layers"] = (case["layers"] + 1) // 2
            case["context"] = (case["context"] + 1) // 2
        return case
    if op == "free":
        case = {"op": op, "rows": _spread(rng, 1, 4095), "context": _spread(rng, 1, 32767),
                "page": rng.choice([16, 32, 64, 128]), "spare": rng.choice([0.01, 0.1, 0.5, 2.0])}
        while work(case)["bytes"] > 2e7:
            case["rows"] = case["rows"] // 2
        return case
    case = {"op": op, "rows": _spread(rng, 1, 255), "context": _spread(rng, 1, 8191), "page": rng.choice([16, 32, 64, 128]),
            "layers": _spread(rng, 1, 32), "kv_heads": rng.choice([1, 2, 8, 16]), "dim": rng.choice([64, 80, 128]),
            "moved": rng.choice([0.0, 0.02, 0.2, 0.45]), "spare": rng.choice([0.5, 1.0]),
            "dtype": rng.choice(["fp16", "bf16"])}
    while _cache_bytes(case, 2 * sum(_pages(case))) > 5e9 or work(case)["bytes"] > 1.4e9:
        case["rows"] = (case["rows"] + 1) // 2
        case["layers"] = (case["layers"] + 1) // 2
        case["context"] = (case["context"] + 1) // 2
    return case


def _chance(case):
    """A case's own random numbers."""
    return random.Random(sum(v for v in case.values() if isinstance(v, int)))


def _lengths(case, n):
    """`n` lengths between a tenth and all of the case's context, the first one whole."""
    r = _chance(case)
    return [case["context"]] + [max(1, int(case["context"] * r.uniform(0.1, 1.0))) for _ in range(n - 1)]


def _pages(case):
    return [-(-n // case["page"]) for n in _lengths(case, case["rows"])]


def _fork_pages(case):
    """(pages that a request's beams share, all its pages) of every request: half of its context is a prompt."""
    shared, every = [], []
    for n in _lengths(case, case["requests"]):
        s = n // 2 // case["page"]
        shared.append(s)
        every.append(s + case["beams"] * (-(-n // case["page"]) - s))
    return shared, every


def _fork_parents(case):
    """Which beams of each request go on, as [requests][beams]: some twice or more, some not at all."""
    r = _chance(case)
    return [[r.randrange(case["beams"]) for _ in range(case["beams"])] for _ in range(case["requests"])]


def _fork_copies(case):
    """(tokens of every page that is copied, in all)."""
    tokens = []
    for n, parents in zip(_lengths(case, case["requests"]), _fork_parents(case)):
        if n % case["page"]:
            tokens += [n % case["page"]] * (len(parents) - len(set(parents)))
    return tokens


def _moves(case):
    return int(case["moved"] * sum(_pages(case)))


def _cache_bytes(case, blocks):
    return 4 * case["layers"] * case["page"] * case["kv_heads"] * case["dim"] * blocks


def _i32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


def _table(blocks, width):
    """int32 [rows, width] of lists of blocks, -1 after them."""
    table = np.full((len(blocks), width), -1, dtype=np.int32)
    for b, row in enumerate(blocks):
        table[b, :len(row)] = row
    return torch.from_numpy(table).cuda()


def _axes(case):
    """The axis of every frequency: a quarter time, the rest height and width, in blocks or taking turns."""
    n = case["rotated"] // 2
    first = n // 4
    left = [first, (n - first + 1) // 2, (n - first) // 2]
    got = []
    if case["cycle"]:
        while len(got) < n:
            for a in range(3):
                if left[a] > 0:
                    left[a] -= 1
                    got.append(a)
    else:
        got = [a for a in range(3) for _ in range(left[a])]
    return _i32(got)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed + 1)
    s = {"op": case["op"]}

    def normal(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)

    if case["op"] == "rotary":
        T, H, K, D, page = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"]
        dtype = DTYPES[case["dtype"]]
        # queries, keys and values are parts of one projection's output row, as the fused qkv layer leaves them
        qkv = normal(T, H + 2 * K, D, dtype=dtype)
        start = int(rng.integers(0, max(1, case["far"] - T)))
        if case["axes"] == 1:
            positions = start + torch.arange(T, device="cuda", dtype=torch.int32)
        else:      # frames of 30 x 40 patches that follow a text
            at = torch.arange(T, device="cuda", dtype=torch.int32)
            positions = start + torch.stack([at // 1200, at // 40 % 30, at % 40])
        base = [1e4, 5e5, 1e6][case["far"] % 3]
        s.update(q=qkv[:, :H], k=qkv[:, H:H + K], v=qkv[:, H + K:], positions=positions.contiguous(),
                 inv_freq=(base ** (-torch.arange(case["rotated"] // 2, dtype=torch.float64) * 2 / case["rotated"]))
                 .float().cuda(), axes=_axes(case) if case["axes"] > 1 else None, pairs=case["pairs"], append=case["append"])
        if case["append"]:
            blocks = -(-T // page) + 2
            perm = torch.from_numpy(rng.permutation(blocks)).cuda()
            at = torch.arange(T, device="cuda")
            s.update(slots=perm[at // page] * page + at % page,
                     k_cache=torch.zeros((blocks, page, K, D), dtype=dtype, device="cuda"),
                     v_cache=torch.zeros((blocks, page, K, D), dtype=dtype, device="cuda"))
        return s
    if case["op"] == "beam":
        B, W, V = case["requests"], case["beams"], case["vocab"]
        logits = normal(B * W, V, dtype=torch.float32).mul_(3)
        if case["masked"]:
            logits[torch.rand(logits.shape, device="cuda", generator=gen) < 0.6] = -torch.inf
        # an end token is now and then among the best
        ends = np.sort(rng.choice(V, case["ends"], replace=False))
        if case["ends"]:
            rows = torch.from_numpy(rng.integers(0, B * W, -(-B * W // 3))).cuda()
            logits[rows, int(ends[0])] = 12.0
        s.update(logits=logits.to(DTYPES[case["dtype"]]), keep=case["keep"],
                 scores=-20 - 3 * torch.rand((B, W), device="cuda", generator=gen),
                 ends=_i32(ends) if case["ends"] else None,
                 history=torch.randint(V, (B * W, case["history"]), device="cuda", generator=gen, dtype=torch.int32))
        return s
    if case["op"] == "free":
        have = [_pages(case)[i] for i in rng.permutation(case["rows"])]
        context = [_lengths(case, case["rows"])[i] for i in np.random.default_rng(seed + 1).permutation(case["rows"])]
        blocks = int(sum(have) * (1 + case["spare"])) + 1
        perm = rng.permutation(blocks).astype(np.int32)
        ends = np.cumsum(have)
        s.update(table=_table([perm[e - n:e] for n, e in zip(have, ends)], max(have) + 2), lens=_i32(context),
                 page=case["page"], blocks=blocks)
        return s
    dtype, shape = DTYPES[case["dtype"]], (case["page"], case["kv_heads"], case["dim"])
    if case["op"] == "fork":
        W, order = case["beams"], rng.permutation(case["requests"])
        lens = [_lengths(case, case["requests"])[i] for i in order]
        shared, every = ([v[i] for i in order] for v in _fork_pages(case))
        parents = [_fork_parents(case)[i] for i in order]
        copies, start = len(_fork_copies(case)), int(rng.integers(0, 5))
        blocks = sum(every) + copies + 8
        perm = rng.permutation(blocks).astype(np.int32)
        rows, at = [], 0
        for n, p, e in zip(lens, shared, every):
            mine = -(-n // case["page"]) - p
            rows += [np.concatenate([perm[at:at + p], perm[at + p + w * mine:at + p + (w + 1) * mine]]) for w in range(W)]
            at += e
        cache = normal(case["layers"], 2, blocks, *shape, dtype=dtype)
        s.update(table=_table(rows, max(len(r) for r in rows) + 2), lens=_i32(np.repeat(lens, W)),
                 parents=_i32([b * W + p for b, ps in enumerate(parents) for p in ps]),
                 # the step's plan has taken the first blocks of the list
                 free=torch.from_numpy(perm[at:].copy()).cuda(), start=_i32([start]), page=case["page"],
                 cache=cache, caches=list(cache.flatten(0, 1).unbind(0)))
        return s
    have = [_pages(case)[i] for i in rng.permutation(case["rows"])]
    context = [_lengths(case, case["rows"])[i] for i in np.random.default_rng(seed + 1).permutation(case["rows"])]
    n, m = sum(have), _moves(case)
    blocks = n + max(m, int(n * case["spare"])) + 1
    used = np.concatenate([rng.choice(n, n - m, replace=False), n + rng.choice(blocks - n, m, replace=False)])
    used = rng.permutation(used).astype(np.int32)
    cache = normal(case["layers"], 2, blocks, *shape, dtype=dtype)
    ends = np.cumsum(have)
    s.update(table=_table([used[e - k:e] for k, e in zip(have, ends)], max(have) + 2), lens=_i32(context),
             page=case["page"], blocks=blocks, cache=cache, caches=list(cache.flatten(0, 1).unbind(0)))
    return s


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def work(case):
    if case["op"] == "rotary":
        T, D = case["tokens"], case["dim"]
        heads = case["heads"] + case["kv_heads"] * (2 if case["append"] else 1)
        return {"bytes": T * (4 * D * heads + 4 * case["axes"] + (8 if case["append"] else 0)) + 4 * case["rotated"],
                "flops": 3 * T * case["rotated"] * (case["heads"] + case["kv_heads"])}
    if case["op"] == "beam":
        size = torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
        B, N = case["requests"], case["requests"] * case["beams"]
        return {"bytes": N * case["vocab"] * size + 8 * B * case["keep"] * case["history"] + 4 * N + 24 * B * case["keep"],
                "flops": 4 * N * case["vocab"]}
    if case["op"] == "fork":
        tokens = _fork_copies(case)
        rows, lens = case["requests"] * case["beams"], _lengths(case, case["requests"])
        width = max(-(-n // case["page"]) for n in lens) + 2
        entries = sum(-(-n // case["page"]) for n in lens) * case["beams"]
        return {"bytes": 8 * case["layers"] * case["kv_heads"] * case["dim"] * sum(tokens) + 4 * entries
                + 4 * rows * width + 16 * rows + 16 * len(tokens), "flops": 0}
    pages = _pages(case)
    if case["op"] == "free":
        return {"bytes": 4 * sum(pages) + 4 * case["rows"] + 4 * (int(sum(pages) * (1 + case["spare"])) + 1), "flops": 0}
    blocks = sum(pages) + max(_moves(case), int(sum(pages) * case["spare"])) + 1
    return {"bytes": 2 * _cache_bytes(case, _moves(case)) + 4 * sum(pages) + 4 * case["rows"] * (max(pages) + 3)
            + 4 * blocks + 8 * _moves(case), "flops": 0}


# ---- the package's operators ----

def _own_rotary(s):
    import bit_weight_quantized_awq_gb300 as awq
    if not s["append"]:
        return awq.rotary(s["q"], s["k"], s["positions"], s["inv_freq"], axes=s["axes"], pairs=s["pairs"])
    q = awq.rotary_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["k_cache"], s["v_cache"], s["slots"],
                          axes=s["axes"], pairs=s["pairs"])
    return q, s["k_cache"], s["v_cache"]


def _own_beam(s):
    import bit_weight_quantized_awq_gb300 as awq
    step = awq.beam_select(s["logits"], s["scores"], s["keep"], end_tokens=s["ends"])
    history, = awq.reorder_states([s["history"]], step.parents.view(-1))
    got = {"scores": step.scores, "parents": step.parents, "tokens": step.tokens, "history": history}
    if s["ends"] is not None:
        got.update(ended_scores=step.ended_scores, ended_parents=step.ended_parents, ended_tokens=step.ended_tokens)
    return got


def _own_fork(s):
    import bit_weight_quantized_awq_gb300 as awq
    f = awq.fork_pages(s["table"], s["lens"], s["parents"], s["free"], s["page"], free_start=s["start"])
    awq.copy_pages(s["caches"], f.src, f.dst, tokens=f.tokens, count=f.count)
    return {"table": f.block_table, "lens": f.lens, "src": f.src, "dst": f.dst, "tokens": f.tokens, "count": f.count,
            "cache": s["cache"]}


def _own_free(s):
    import bit_weight_quantized_awq_gb300 as awq
    f = awq.free_pages(s["table"], s["lens"], s["page"], s["blocks"])
    return f.free_blocks, f.counts


def _own_compact(s):
    import bit_weight_quantized_awq_gb300 as awq
    c = awq.compact_pages(s["table"], s["lens"], s["page"], s["blocks"])
    awq.copy_pages(s["caches"], c.src, c.dst, count=c.count)
    return {"table": c.block_table, "map": c.block_map, "src": c.src, "dst": c.dst, "count": c.count, "cache": s["cache"]}


_own = {"rotary": _own_rotary, "beam": _own_beam, "fork": _own_fork, "free": _own_free, "compact": _own_compact}


# ---- the plain forms ----

def _plain_rotary(s):
    f, axes, T = s["inv_freq"].double(), s["axes"], s["q"].shape[0]
    # far positions: a product in 32 bits would lose the angle
    at = s["positions"].double()
    angle = at[:, None] * f if axes is None else at[axes.long()].T * f
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    n = f.numel()

    def turned(x):
        y = x.float()
        r, rest = y[..., :2 * n], y[..., 2 * n:]
        if s["pairs"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :n], r[..., n:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, rest], -1).to(x.dtype)

    q, k = turned(s["q"]), turned(s["k"])
    if not s["append"]:
        return q, k
    s["k_cache"].flatten(0, 1)[s["slots"]] = k
    s["v_cache"].flatten(0, 1)[s["slots"]] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _plain_beam(s):
    logits, scores, W = s["logits"], s["scores"], s["keep"]
    B, V = scores.shape[0], logits.shape[1]
    E = 0 if s["ends"] is None else s["ends"].numel()
    # the log-sum-exp in 64 bits, since the order of nearly equal candidates hangs on it
    x = logits.float() + 0.0
    top = x.amax(-1, keepdim=True)
    lse = torch.log(torch.exp((x - top).double()).sum(-1)) + top[:, 0].double()
    # the best of each row by logit, then by the lowest token: keys that are all different
    bits = x.view(torch.int32)
    keys = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32 + (2 ** 32 - 1 - torch.arange(V, device=x.device))
    best = torch.topk(keys, min(V, W + E), dim=-1).values
    token = 2 ** 32 - 1 - (best & 0xFFFFFFFF)
    score = scores.view(-1, 1).double() + (x.gather(1, token).double() - lse[:, None])
    score, token = score.view(B, -1), token.view(B, -1)
    score, order = torch.sort(score, dim=-1, descending=True, stable=True)
    token = token.gather(1, order)
    row = order // best.shape[1] + torch.arange(B, device=x.device)[:, None] * scores.shape[1]
    good = score > -torch.inf
    end = torch.zeros_like(good) if E == 0 else (token[..., None] == s["ends"]).any(-1)

    def first(mask):
        """The first W of a request's candidates that `mask` has."""
        at = torch.cumsum(mask, -1) - 1
        at = torch.where(mask & (at < W), at, W)
        return [torch.full((B, W + 1), none, dtype=v.dtype, device=x.device).scatter_(1, at, v)[:, :W]
                for v, none in ((score.float(), -torch.inf), (row.int(), -1), (token.int(), -1))]

    got = dict(zip(("scores", "parents", "tokens"), first(good & ~end)))
    if E:
        rank = torch.arange(score.shape[1], device=x.device)
        got.update(zip(("ended_scores", "ended_parents", "ended_tokens"), first(good & end & (rank < W))))
    parents = got["parents"].flatten().long()
    got["history"] = torch.where(parents[:, None] >= 0, s["history"][parents.clamp(min=0)], 0)
    return got


def _plain_fork(s):
    table, page, p = s["table"], s["page"], s["parents"].long()
    R, width = table.shape
    r = torch.arange(p.numel(), device=table.device)
    lens = s["lens"].long()[p]
    have, part = (lens + page - 1) // page, lens % page
    first = torch.full((R,), p.numel(), device=table.device).scatter_reduce(0, p, r, "amin")
    need = (part > 0) & (first[p] != r)
    rank = torch.cumsum(need, 0) - 1
    fresh = s["free"][(s["start"].long() + rank).clamp(0, s["free"].numel() - 1)]
    j = torch.arange(width, device=table.device)
    last = j == have[:, None] - 1
    new = torch.where(j < have[:, None], table[p], -1)
    old = table[p].gather(1, (have[:, None] - 1).clamp(min=0))[:, 0]
    new = torch.where(last & need[:, None], fresh[:, None], new)

    def listed_up(v):
        return torch.full((p.numel() + 1,), -1, dtype=torch.int32, device=v.device).scatter_(
            0, torch.where(need, rank, p.numel()), v.int())[:-1]

    got = {"table": new, "lens": lens.int(), "src": listed_up(old), "dst": listed_up(fresh), "tokens": listed_up(part),
           "count": need.sum().int().view(1), "cache": s["cache"]}
    src, dst, tokens = old[need].long(), fresh[need].long(), part[need]
    kept = (torch.arange(page, device=table.device) < tokens[:, None])[:, :, None, None]
    s["cache"][:, :, dst] = torch.where(kept, s["cache"][:, :, src], s["cache"][:, :, dst])
    return got


def _used(s):
    table, n = s["table"], s["blocks"]
    have = (s["lens"].long() + s["page"] - 1) // s["page"]
    named = torch.where(torch.arange(table.shape[1], device=table.device) < have[:, None], table, n)
    used = torch.zeros(n + 1, dtype=torch.bool, device=table.device)
    used[named.long().flatten()] = True
    return used[:n]


def _in_order(mask, values, size):
    """int32 [size]: the values where `mask` is set, in their order, then -1."""
    at = torch.where(mask, torch.cumsum(mask, 0) - 1, size)
    return torch.full((size + 1,), -1, dtype=torch.int32, device=mask.device).scatter_(0, at, values.int())[:size]


def _plain_free(s):
    used = _used(s)
    block = torch.arange(s["blocks"], device=used.device)
    count = used.sum()
    return _in_order(~used, block, s["blocks"]), torch.stack([s["blocks"] - count, count]).int()


def _plain_compact(s):
    used = _used(s)
    block, n = torch.arange(s["blocks"], device=used.device), used.sum()
    moves = used & (block >= n)
    holes = _in_order(~used & (block < n), block, s["blocks"])
    to = holes[(torch.cumsum(moves, 0) - 1).clamp(min=0)]
    renamed = torch.where(used, torch.where(moves, to, block.int()), -1)
    table = s["table"]
    have = (s["lens"].long() + s["page"] - 1) // s["page"]
    inside = torch.arange(table.shape[1], device=table.device) < have[:, None]
    table = torch.where(inside, renamed[table.clamp(min=0).long()], -1)
    half = s["blocks"] // 2
    got = {"table": table, "map": renamed, "src": _in_order(moves, block, half), "dst": _in_order(moves, to, half),
           "count": moves.sum().int().view(1), "cache": s["cache"]}
    s["cache"][:, :, to[moves].long()] = s["cache"][:, :, block[moves]]
    return got


_plain = {"rotary": _plain_rotary, "beam": _plain_beam, "fork": _plain_fork, "free": _plain_free, "compact": _plain_compact}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    if case["op"] == "rotary":
        return _exact_rotary(prepare(case, seed))
    if case["op"] == "beam":
        return _exact_beam(prepare(case, seed))
    return None      # whole numbers and copies


def _exact_rotary(s):
    n, pairs = s["inv_freq"].numel(), s["pairs"]
    rows = s["positions"].view(-1, s["positions"].shape[-1])
    which = [0] * n if s["axes"] is None else s["axes"].tolist()

    def turned(x):
        y = x.double()
        out = y.clone()
        for i, a in enumerate(which):
            turn = torch.polar(torch.ones(rows.shape[1], dtype=torch.float64, device=y.device),
                               rows[a].double() * s["inv_freq"][i].double())
            first, second = (2 * i, 2 * i + 1) if pairs else (i, i + n)
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            out[..., first], out[..., second] = z.real, z.imag
        return out

    q, k = turned(s["q"]), turned(s["k"])
    if not s["append"]:
        return q, k
    caches = []
    for x, cache in ((k, s["k_cache"]), (s["v"].double(), s["v_cache"])):
        made = torch.zeros(cache.shape, dtype=torch.float64, device=cache.device)
        made.view(-1, *cache.shape[2:])[s["slots"]] = x
        caches.append(made)
    return q, *caches


def _exact_beam(s):
    B, W = s["scores"].shape
    keep, ends = s["keep"], set() if s["ends"] is None else set(s["ends"].tolist())
    live, ended = np.full((B, keep), -np.inf), np.full((B, keep), -np.inf)
    for b in range(B):
        x = s["logits"][b * W:(b + 1) * W].double()
        every = (s["scores"][b].double()[:, None] + torch.log_softmax(x, -1)).flatten()
        # no more than these can matter: the kept ones, and every row's end tokens before them
        best, at = torch.sort(every, descending=True, stable=True)
        best, at = (v[:keep + W * len(ends)].tolist() for v in (best, at))
        n = m = 0
        for rank, (score, flat) in enumerate(zip(best, at)):
            if score == -np.inf:
                break
            if flat % x.shape[1] in ends:
                if rank < keep:
                    ended[b, m] = score
                    m += 1
            elif n < keep:
                live[b, n] = score
                n += 1
    got = {"scores": torch.from_numpy(live), "parents": None, "tokens": None, "history": None}
    if ends:
        got.update(ended_scores=torch.from_numpy(ended), ended_parents=None, ended_tokens=None)
    return got
