"""Measured cases of the serving operators: ``paged_plan``, ``kv_append``,
``tree_attention`` and ``process_logits``.

``run`` computes a case with the package's operators where ``own`` is true and
with elementary torch operations in 32 bits where it is false; ``exact``
computes the same from the definitions in 64 bits. ``lengths`` gives a case's
request lengths; a seed changes their order, never their sum, so ``work`` is a
function of the case alone.
"""
import random

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token each for a full decode batch: pure launch latency
        {"name": "plan_decode_b256", "op": "plan", "requests": 256, "new": 1, "context": 4096, "page": 16,
         "tree": False},
        # drafted trees of up to 60 nodes for 64 requests: masks and positions as well
        {"name": "plan_tree_b64", "op": "plan", "requests": 64, "new": 60, "context": 8192, "page": 32,
         "tree": True},
        # the drafted tokens of a small batch
        {"name": "append_tree_b16", "op": "append", "requests": 16, "new": 33, "context": 2048, "page": 16,
         "kv_heads": 8, "dim": 128, "dtype": "fp16"},
        # prompts being filled in, 32 heads of their own
        {"name": "append_prompt_b9", "op": "append", "requests": 9, "new": 2048, "context": 512, "page": 64,
         "kv_heads": 32, "dim": 128, "dtype": "bf16"},
        # one request, one token, a short cache: latency (a 4096-wide layer's 32 heads)
        {"name": "attention_one_b1", "op": "attention", "requests": 1, "new": 1, "context": 500, "page": 16,
         "heads": 32, "kv_heads": 32, "dim": 128, "dtype": "fp16", "tree": False},
        # plain decode of a large batch with grouped heads (an 8192-wide layer's 64 / 8): the cache's bytes
        {"name": "attention_decode_b64", "op": "attention", "requests": 64, "new": 1, "context": 8192, "page": 16,
         "heads": 64, "kv_heads": 8, "dim": 128, "dtype": "fp16", "tree": False},
        # speculative decoding of a mid-size batch, small trees
        {"name": "attention_tree_b16", "op": "attention", "requests": 16, "new": 13, "context": 6000, "page": 64,
         "heads": 64, "kv_heads": 8, "dim": 128, "dtype": "bf16", "tree": True},
        # one long document, a tree of 26 nodes: the cache split along its length
        {"name": "attention_tree_long", "op": "attention", "requests": 1, "new": 26, "context": 131072, "page": 32,
         "heads": 32, "kv_heads": 8, "dim": 64, "dtype": "bf16", "tree": True},
        # large trees, grouped heads: hundreds of rows a key-value head, the tensor cores' work
        {"name": "attention_tree_b12_wide", "op": "attention", "requests": 12, "new": 64, "context": 16384,
         "page": 128, "heads": 64, "kv_heads": 8, "dim": 128, "dtype": "fp16", "tree": True},
        # one row, a small vocabulary: latency
        {"name": "logits_one", "op": "logits", "requests": 1, "new": 1, "vocab": 32000, "history": 700,
         "bias": 16, "dtype": "fp16", "grammar": True},
        # a decode batch with long histories
        {"name": "logits_decode_b64", "op": "logits", "requests": 64, "new": 1, "vocab": 131072, "history": 4000,
         "bias": 300, "dtype": "fp32", "grammar": True},
        # every node of 16 requests' trees has its logits processed
        {"name": "logits_tree_b16", "op": "logits", "requests": 16, "new": 48, "vocab": 100000, "history": 2500,
         "bias": 64, "dtype": "bf16", "grammar": True},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm, odd when above 64."""
    v = int(round(low * (high / low) ** rng.random()))
    return v if v <= 64 else min(high, v) - (1 - min(high, v) % 2)


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "attention", "logits", "logits"])
    if op == "plan":
        tree = rng.random() < 0.5
        return {"op": op, "requests": _spread(rng, 1, 256), "new": _spread(rng, 2, 100) if tree else _spread(rng, 1, 400),
                "context": _spread(rng, 1, 8191), "page": rng.choice([16, 32, 64, 128]), "tree": tree}
    if op == "append":
        case = {"op": op, "requests": _spread(rng, 1, 64), "new": _spread(rng, 1, 2047), "context": _spread(rng, 1, 2047),
                "page": rng.choice([16, 32, 64, 128]), "kv_heads": rng.choice([1, 4, 8, 32]),
                "dim": rng.choice([64, 80, 96, 128]), "dtype": rng.choice(["fp16", "bf16"])}
        while work(case)["bytes"] > 3e8:
            case["requests"] = max(1, case["requests"] // 2)
            case["new"] = case["new"] // 2 + 1
        return case
    if op == "attention":
        kv_heads, group = rng.choice([(32, 1), (8, 4), (8, 8), (4, 7), (1, 16), (2, 5)])
        new = rng.choice([1, _spread(rng, 2, 64), _spread(rng, 2, 64)])
        case = {"op": op, "requests": _spread(rng, 1, 64), "new": new, "context": _spread(rng, 17, 131071),
                "page": rng.choice([16, 32, 64, 128]), "heads": kv_heads * group, "kv_heads": kv_heads,
                "dim": rng.choice([64, 128, 128, 96]), "dtype": rng.choice(["fp16", "bf16"]), "tree": new > 1}
        while work(case)["bytes"] > 1.2e9 or work(case)["flops"] > 4.5e11 or _padded(case) > 6e9:
            if case["requests"] > 4:
                case["requests"] //= 2
            else:
                case["context"] = case["context"] // 4 * 2 + 1
        return case
    case = {"op": op, "requests": _spread(rng, 1, 128), "new": _spread(rng, 1, 48), "vocab": _spread(rng, 20000, 160001),
            "history": _spread(rng, 1, 8191), "bias": rng.choice([0, 1, 40, 299]),
            "dtype": rng.choice(["fp16", "bf16", "fp32"]), "grammar": rng.random() < 0.7}
    while work(case)["bytes"] > 3e8:
        case["requests"] = (case["requests"] + 1) // 2
        case["new"] = (case["new"] + 1) // 2
    return case


def _padded(case):
    """Bytes of the plain form's padded keys, values and scores."""
    rows = case["requests"] * (case["context"] + case["new"])
    return 4 * rows * (2 * case["kv_heads"] * case["dim"] + case["new"] * case["heads"])


def lengths(case):
    """(context, new) of every request: between a tenth and all of the case's lengths, the first one whole."""
    r = random.Random(sum(v for v in case.values() if isinstance(v, int)))
    ctx, new = [case.get("context", 0)], [case["new"]]
    for _ in range(case["requests"] - 1):
        ctx.append(max(1, int(case.get("context", 0) * r.uniform(0.1, 1.0))))
        new.append(max(1, int(case["new"] * r.uniform(0.5, 1.0))))
    return ctx, new


def _histories(case):
    """(length, prompt part) of every request's history."""
    r = random.Random(case["history"] * 131 + case["requests"])
    got = []
    for i in range(case["requests"]):
        n = case["history"] if i == 0 else max(1, int(case["history"] * r.uniform(0.1, 1.0)))
        got.append((n, int(n * r.uniform(0.0, 0.9))))
    return got


def _shuffled(case, seed):
    ctx, new = lengths(case)
    order = np.random.default_rng(seed).permutation(len(ctx))
    return [ctx[i] for i in order], [new[i] for i in order]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cumulative(values):
    return _i32([0] + list(np.cumsum(values)))


def _parents(rng, new):
    """A random forest for every request: a node's parent is any earlier node or the context's last token."""
    return np.concatenate([np.floor(rng.random(n) * (np.arange(n) + 1)).astype(np.int32) - 1 for n in new])


def _node_masks(parents, new, words):
    """int32 [tokens, words]: bit j of a node's row is set if j is the node or one of its ancestors."""
    out = np.zeros((sum(new), words), dtype=np.uint32)
    at = 0
    for n in new:
        for i in range(n):
            p = parents[at + i]
            if p >= 0:
                out[at + i] = out[at + p]
            out[at + i, i // 32] |= np.uint32(1 << (i % 32))
        at += n
    return torch.from_numpy(out.view(np.int32)).cuda()


def _tables(rng, ctx, extra, page):
    """(block table with the blocks of `ctx + extra` tokens and -1 after them, number of blocks in the cache)."""
    have = [-(-(c + e) // page) for c, e in zip(ctx, extra)]
    total = sum(have) + 7
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(ctx), max(have) + 4), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), total


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed + 1)
    ctx, new = _shuffled(case, seed)
    s = {"case": case, "op": case["op"]}

    def normal(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)

    if case["op"] == "plan":
        page = case["page"]
        width = -(-max(c + n for c, n in zip(ctx, new)) // page) + 3
        have = [-(-c // page) for c in ctx]
        free = sum(-(-n // page) + 1 for n in new)
        perm = rng.permutation(sum(have) + free).astype(np.int32)
        table = np.full((len(ctx), width), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(have):
            table[b, :n] = perm[at:at + n]
            at += n
        s.update(context_lens=_i32(ctx), new_lens=_i32(new), block_table=torch.from_numpy(table).cuda(),
                 free_blocks=torch.from_numpy(perm[at:].copy()).cuda(), page=page, tokens=sum(new),
                 words=-(-case["new"] // 32) if case["tree"] else 0,
                 parents=torch.from_numpy(_parents(rng, new)).cuda() if case["tree"] else None)
        return s
    if case["op"] == "append":
        dtype = DTYPES[case["dtype"]]
        table, blocks = _tables(rng, ctx, new, case["page"])
        at = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)]).cuda()
        req = torch.repeat_interleave(torch.arange(len(ctx)), torch.tensor(new)).cuda()
        slots = table[req, at // case["page"]].long() * case["page"] + at % case["page"]
        heads, dim = case["kv_heads"], case["dim"]
        # keys and values are parts of one projection's output row, as the fused qkv layer leaves them
        qkv = normal(sum(new), 3 * heads, dim, dtype=dtype)
        s.update(k=qkv[:, heads:2 * heads], v=qkv[:, 2 * heads:], slots=slots,
                 k_cache=torch.zeros((blocks, case["page"], heads, dim), dtype=dtype, device="cuda"),
                 v_cache=torch.zeros((blocks, case["page"], heads, dim), dtype=dtype, device="cuda"))
        return s
    if case["op"] == "attention":
        dtype = DTYPES[case["dtype"]]
        table, blocks = _tables(rng, ctx, new, case["page"])
        words = -(-case["new"] // 32)
        s.update(q=normal(sum(new), case["heads"], case["dim"], dtype=dtype),
                 k_cache=normal(blocks, case["page"], case["kv_heads"], case["dim"], dtype=dtype),
                 v_cache=normal(blocks, case["page"], case["kv_heads"], case["dim"], dtype=dtype),
                 block_table=table, context_lens=_i32(ctx), cu_new=_cumulative(new), scale=case["dim"] ** -0.5,
                 max_new=max(new), max_context=max(ctx),
                 tree_mask=_node_masks(_parents(rng, new), new, words) if case["tree"] else None)
        return s
    # logits: histories with a head of frequent tokens, per-request settings, tree rows with their drafted tokens
    V, B, rows = case["vocab"], case["requests"], sum(new)
    hist = [_histories(case)[i] for i in np.random.default_rng(seed).permutation(B)]
    total = sum(n for n, _ in hist)
    bias = [np.sort(rng.choice(V, size=case["bias"], replace=False)) for _ in range(B)]
    words = -(-case["new"] // 32)
    s.update(logits=normal(rows, V, dtype=torch.float32).mul_(4).to(DTYPES[case["dtype"]]),
             row_request=torch.repeat_interleave(torch.arange(B, dtype=torch.int32), torch.tensor(new)).cuda(),
             history=torch.from_numpy((V * rng.random(total) ** 3).astype(np.int32)).cuda(),
             history_offsets=_cumulative([n for n, _ in hist]), prompt_lens=_i32([p for _, p in hist]),
             repetition=torch.from_numpy(rng.uniform(1.0, 1.4, B).astype(np.float32)).cuda(),
             frequency=torch.from_numpy(rng.uniform(0.0, 0.5, B).astype(np.float32)).cuda(),
             presence=torch.from_numpy(rng.uniform(0.0, 0.8, B).astype(np.float32)).cuda(),
             draft_tokens=torch.from_numpy((V * rng.random(rows) ** 3).astype(np.int32)).cuda(),
             cu_new=_cumulative(new), tree_mask=_node_masks(_parents(rng, new), new, words),
             bias_tokens=torch.from_numpy(np.concatenate(bias).astype(np.int32)).cuda() if case["bias"] else None,
             bias_values=torch.from_numpy(rng.normal(0, 2, B * case["bias"]).astype(np.float32)).cuda()
             if case["bias"] else None,
             bias_offsets=_i32([i * case["bias"] for i in range(B + 1)]) if case["bias"] else None,
             # a grammar state's mask for every row: most words wholly forbidden, some wholly or partly allowed
             grammar_mask=torch.from_numpy(np.where(
                 rng.random((rows, -(-V // 32))) < 0.5, 0,
                 rng.integers(-2 ** 31, 2 ** 31, (rows, -(-V // 32)))).astype(np.int32)).cuda()
             if case["grammar"] else None, max_new=case["new"])
    return s


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def work(case):
    ctx, new = lengths(case)
    B, T = len(ctx), sum(new)
    if case["op"] == "plan":
        page = case["page"]
        blocks = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        words = -(-case["new"] // 32) if case["tree"] else 0
        return {"bytes": 12 * B + 4 + T * (16 + 4 * words + (4 if case["tree"] else 0)) + 8 * blocks + 4 * B, "flops": 0}
    if case["op"] == "append":
        return {"bytes": T * (8 * case["kv_heads"] * case["dim"] + 8), "flops": 0}
    if case["op"] == "attention":
        D, H, K, page = case["dim"], case["heads"], case["kv_heads"], case["page"]
        blocks = sum(-(-(c + n) // page) for c, n in zip(ctx, new))
        keys = sum(c + n for c, n in zip(ctx, new))
        # every row meets its whole context and, of the drafted keys, at least itself
        pairs = sum(n * (c + 1) for c, n in zip(ctx, new))
        masks = 4 * T * -(-case["new"] // 32) if case["tree"] else 0
        return {"bytes": 4 * K * D * keys + 4 * T * H * D + 4 * blocks + 8 * B + masks, "flops": 4 * D * H * pairs}
    size = torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
    V = case["vocab"]
    return {"bytes": T * V * 2 * size + (T * -(-V // 32) * 4 if case["grammar"] else 0)
            + 4 * sum(n for n, _ in _histories(case)) + 8 * B * case["bias"] + 28 * B, "flops": 0}


# ---- the package's operators ----

def _own_plan(s):
    import bit_weight_quantized_awq_gb300 as awq
    p = awq.paged_plan(s["context_lens"], s["new_lens"], s["block_table"], s["free_blocks"], s["page"], s["tokens"],
                       parents=s["parents"], mask_words=s["words"])
    got = {"cu_new": p.cu_new, "slots": p.slot_map, "positions": p.positions, "request": p.token_request,
           "table": s["block_table"], "counts": p.counts}
    if s["words"]:
        got["mask"] = p.tree_mask
    return got


def _own_append(s):
    import bit_weight_quantized_awq_gb300 as awq
    awq.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
    return s["k_cache"], s["v_cache"]


def _own_attention(s):
    import bit_weight_quantized_awq_gb300 as awq
    return awq.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["context_lens"], s["cu_new"],
                              scale=s["scale"], max_new=s["max_new"], max_context=s["max_context"],
                              tree_mask=s["tree_mask"])


def _own_logits(s):
    import bit_weight_quantized_awq_gb300 as awq
    return awq.process_logits(
        s["logits"], row_request=s["row_request"], history=s["history"], history_offsets=s["history_offsets"],
        prompt_lens=s["prompt_lens"], repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
        draft_tokens=s["draft_tokens"], cu_new=s["cu_new"], tree_mask=s["tree_mask"], bias_tokens=s["bias_tokens"],
        bias_values=s["bias_values"], bias_offsets=s["bias_offsets"], grammar_mask=s["grammar_mask"])


_own = {"plan": _own_plan, "append": _own_append, "attention": _own_attention, "logits": _own_logits}


# ---- the plain forms ----

def _bits(mask, width):
    """bool [tokens, width]: the first `width` bits of every row of an int32 mask."""
    j = torch.arange(width, device=mask.device)
    return (mask[:, j // 32] >> (j % 32).int()) & 1 != 0


def _plain_plan(s):
    ctx, new, table, page, T = s["context_lens"].long(), s["new_lens"].long(), s["block_table"], s["page"], s["tokens"]
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    have = (ctx + page - 1) // page
    need = (ctx + new + page - 1) // page - have
    base = torch.cumsum(need, 0) - need
    j = torch.arange(table.shape[1], device=table.device) - have[:, None]
    fresh = (j >= 0) & (j < need[:, None])
    at = (base[:, None] + j).clamp(0, s["free_blocks"].numel() - 1)
    table.copy_(torch.where(fresh, s["free_blocks"][at], table))
    token = torch.arange(T, device=table.device)
    req = torch.searchsorted(cu, token, right=True) - 1
    local = token - cu[req]
    key = ctx[req] + local
    slots = table[req, key // page].long() * page + key % page
    counts = torch.stack([cu[-1], need.sum()]).int()
    got = {"cu_new": cu.int(), "slots": slots, "request": req.int(), "table": table, "counts": counts}
    if not s["words"]:
        got["positions"] = key.int()
        return got
    # ancestors by doubling: `seen` holds a node's ancestors 2^r steps up, `up` the node 2^r steps up
    n = 32 * s["words"]
    up = torch.where(s["parents"] >= 0, cu[req] + s["parents"], T)
    seen = torch.zeros((T + 1, n), dtype=torch.bool, device=table.device)
    seen[token, local] = True
    up = torch.cat([up, up.new_full((1,), T)])
    for _ in range((n - 1).bit_length()):
        seen = seen | seen[up]
        up = up[up]
    weight = 1 << torch.arange(32, device=table.device)
    words = (seen[:T].view(T, s["words"], 32).long() * weight).sum(-1)
    got["mask"] = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
    got["positions"] = (ctx[req] + seen[:T].sum(-1) - 1).int()
    return got


def _plain_append(s):
    heads, dim = s["k"].shape[1:]
    s["k_cache"].view(-1, heads, dim)[s["slots"]] = s["k"]
    s["v_cache"].view(-1, heads, dim)[s["slots"]] = s["v"]
    return s["k_cache"], s["v_cache"]


def _plain_attention(s):
    q, cu, ctx = s["q"], s["cu_new"].long(), s["context_lens"].long()
    T, H, D = q.shape
    page, K = s["k_cache"].shape[1:3]
    B, N = ctx.numel(), s["max_new"]
    new = cu[1:] - cu[:-1]
    blocks = -(-(s["max_context"] + N) // page)
    table = s["block_table"][:, :blocks].long().clamp(min=0)
    L = table.shape[1] * page
    k = s["k_cache"][table].view(B, L, K, D).float()
    v = s["v_cache"][table].view(B, L, K, D).float()
    key = torch.arange(L, device=q.device)
    v = torch.where((key < (ctx + new)[:, None])[:, :, None, None], v, 0.0)
    t = torch.arange(N, device=q.device)
    row = (cu[:-1, None] + t).clamp(max=T - 1)                    # [B, N]
    drafted = key - ctx[:, None]                                  # [B, L]
    at = drafted.clamp(0, N - 1)
    if s["tree_mask"] is None:
        bit = at[:, None, :] <= t[:, None]
    else:
        bit = _bits(s["tree_mask"], N)[row].gather(2, at[:, None, :].expand(B, N, L))
    seen = (drafted < 0)[:, None, :] | ((drafted >= 0) & (drafted < new[:, None]))[:, None, :] & bit    # [B, N, L]
    qp = q.float()[row].view(B, N, K, H // K, D)
    scores = torch.einsum("bnkgd,blkd->bkngl", qp, k) * s["scale"]
    scores = torch.where(seen[:, None, :, None, :], scores, -torch.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.einsum("bkngl,blkd->bnkgd", p, v)
    token = torch.arange(T, device=q.device)
    req = torch.searchsorted(cu, token, right=True) - 1
    return out[req, token - cu[req]].reshape(T, H, D).to(q.dtype)


def _plain_logits(s):
    logits, req = s["logits"], s["row_request"].long()
    R, V = logits.shape
    B = s["prompt_lens"].numel()
    off = s["history_offsets"].long()
    at = torch.arange(s["history"].numel(), device=logits.device)
    owner = torch.searchsorted(off, at, right=True) - 1
    prompt = at - off[owner] < s["prompt_lens"][owner]
    flat = owner * V + s["history"]
    one = torch.ones_like(flat, dtype=torch.int32)
    said = torch.zeros(B * V, dtype=torch.int32, device=logits.device).scatter_add_(0, flat, one * ~prompt)
    known = torch.zeros(B * V, dtype=torch.int32, device=logits.device).scatter_add_(0, flat, one)
    count, known = said.view(B, V)[req], known.view(B, V)[req]
    n = s["max_new"]
    first = s["cu_new"].long()[req]
    node = (first[:, None] + torch.arange(n, device=logits.device)).clamp(max=R - 1)
    path = _bits(s["tree_mask"], n).int()
    count.scatter_add_(1, s["draft_tokens"].long()[node], path)
    known.scatter_add_(1, s["draft_tokens"].long()[node], path)
    x = logits.float()
    rep = s["repetition"][req][:, None]
    x = torch.where(known > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][req][:, None] * count - s["presence"][req][:, None] * (count > 0)
    if s["bias_tokens"] is not None:
        boff = s["bias_offsets"].long()
        bowner = torch.searchsorted(boff, torch.arange(s["bias_tokens"].numel(), device=x.device), right=True) - 1
        dense = torch.zeros(B * V, device=x.device).scatter_add_(0, bowner * V + s["bias_tokens"], s["bias_values"])
        x = x + dense.view(B, V)[req]
    if s["grammar_mask"] is not None:
        x = torch.where(_bits(s["grammar_mask"], V), x, -torch.inf)
    return x.to(logits.dtype)


_plain = {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention, "logits": _plain_logits}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(prepare(case, seed))
    if case["op"] == "logits":
        return _exact_logits(prepare(case, seed))
    return None      # whole numbers and copies


def _exact_attention(s):
    q, page = s["q"].double(), s["k_cache"].shape[1]
    group = q.shape[1] // s["k_cache"].shape[2]
    cu, ctx = s["cu_new"].tolist(), s["context_lens"].tolist()
    out = torch.zeros_like(q)
    for b, c in enumerate(ctx):
        n = cu[b + 1] - cu[b]
        blocks = s["block_table"][b, :-(-(c + n) // page)].long()
        k = s["k_cache"][blocks].flatten(0, 1)[:c + n]
        v = s["v_cache"][blocks].flatten(0, 1)[:c + n]
        seen = torch.ones((n, c + n), dtype=torch.bool, device=q.device)
        if s["tree_mask"] is None:
            seen[:, c:] = torch.ones((n, n), device=q.device).tril().bool()
        else:
            mask = s["tree_mask"][cu[b]:cu[b + 1]].cpu().numpy().view(np.uint32)
            bits = np.unpackbits(mask.view(np.uint8), axis=1, bitorder="little")[:, :n]
            seen[:, c:] = torch.from_numpy(bits.astype(bool)).to(q.device)
        for h in range(k.shape[1]):
            rows = q[cu[b]:cu[b + 1], h * group:(h + 1) * group].transpose(0, 1)      # [group, n, D]
            a = (rows @ k[:, h].double().T) * s["scale"]
            a = a.masked_fill(~seen, -torch.inf).softmax(-1).masked_fill(~seen, 0.0)
            out[cu[b]:cu[b + 1], h * group:(h + 1) * group] = (a @ v[:, h].double()).transpose(0, 1)
    return out


def _exact_logits(s):
    V = s["logits"].shape[1]
    get = lambda name: None if s[name] is None else s[name].cpu().numpy()  # noqa: E731
    req, hist, off, prompt = get("row_request"), get("history"), get("history_offsets"), get("prompt_lens")
    rep, freq, pres = (get(n).astype(np.float64) for n in ("repetition", "frequency", "presence"))
    draft, cu, mask = get("draft_tokens"), get("cu_new"), get("tree_mask").view(np.uint32)
    bo, bt, bv, gm = get("bias_offsets"), get("bias_tokens"), get("bias_values"), get("grammar_mask")
    out = s["logits"].double()
    for r, b in enumerate(req):
        h = hist[off[b]:off[b + 1]]
        node = np.unpackbits(mask[r].view(np.uint8), bitorder="little").nonzero()[0]
        path = draft[cu[b] + node]
        said = np.bincount(np.concatenate([h[prompt[b]:], path]), minlength=V)
        known = np.unique(np.concatenate([h, path]))
        x = out[r].cpu().numpy().copy()
        x[known] = np.where(x[known] > 0, x[known] / rep[b], x[known] * rep[b])
        x -= freq[b] * said + pres[b] * (said > 0)
        if bt is not None:
            np.add.at(x, bt[bo[b]:bo[b + 1]], bv[bo[b]:bo[b + 1]].astype(np.float64))
        if gm is not None:
            allowed = np.unpackbits(gm[r].view(np.uint32).view(np.uint8), bitorder="little")[:V]
            x[allowed == 0] = -np.inf
        out[r] = torch.from_numpy(x).cuda()
    return out
