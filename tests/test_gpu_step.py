"""GPU tests of the decoding step's operators (paged_plan, kv_append,
tree_attention, process_logits) against 64-bit references on the CPU.

Tolerances, from the formats (u = 2^-11 for fp16, 2^-8 for bf16, half a unit in
the last place relative to the value):
  attention  |out - ref| <= u |ref| + (u + 2^-13) sum_j w_j |v_j| + 2^-24: the
             output's rounding; each softmax weight's rounding to q's type and
             the fp32 errors of scores, exponentials and sums (2^-13 covers
             a few thousand fp32 additions); fp16's subnormal step.
             |lse - ref| <= 2^-13 (1 + |ref|) for the fp32 part.
  logits     a few fp32 roundings and one to the output's type:
             |out - ref| <= (u + 2^-21) |ref| + 2^-20 (1 + |x| + penalties) with
             u = 0 for fp32.
Whole numbers and copies are compared for equality.
"""
import numpy as np
import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
import step_reference as ref
from bit_weight_quantized_awq_gb300 import Status

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


@pytest.fixture(autouse=True)
def _status(gpu):
    """Every test starts and ends with a clean device status."""
    awq.awq_last_device_status(None)
    yield
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


def i32(values):
    return torch.tensor(np.asarray(values, dtype=np.int64), dtype=torch.int64).to(torch.int32).cuda()


def forest(rng, new):
    """Parents of random forests: any earlier node, or -1."""
    return np.concatenate([np.floor(rng.random(n) * (np.arange(n) + 1)).astype(np.int64) - 1 for n in new]
                          + [np.zeros(0, dtype=np.int64)])


def tables(rng, ctx, new, page, spare=3):
    have = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    total = sum(have) + spare
    perm = rng.permutation(total)
    table = np.full((len(ctx), max(have + [1]) + 2), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


# ---------------------------------------------------------------- plan

@pytest.mark.parametrize("ctx,new,page", [
    ([0], [1], 16), ([15], [1], 16), ([16], [1], 16), ([31, 0, 5], [2, 0, 40], 16), ([0, 0], [0, 0], 32),
    ([100, 7, 64, 63, 65, 1], [33, 1, 64, 1, 2, 128], 64), ([5] * 700, [1, 2, 0, 3, 5, 1, 1] * 100, 16),
    ([1000], [5000], 128), (list(range(1300)), [1] * 1300, 1024)])
@pytest.mark.parametrize("tree", [False, True])
def test_plan_matches_the_reference(ctx, new, page, tree):
    rng = np.random.default_rng(len(ctx) + page)
    words = -(-max(new + [1]) // 32) if tree or max(new) <= 200 else 0
    have = [-(-c // page) for c in ctx]
    need = sum(-(-(c + n) // page) for c, n in zip(ctx, new)) - sum(have)
    perm = rng.permutation(sum(have) + need + 5)
    width = max(-(-(c + n) // page) for c, n in zip(ctx, new)) + 2
    table = np.full((len(ctx), width), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = perm[at:at + n]
        at += n
    parents = forest(rng, new) if tree else None
    cu, want_table, slots, positions, request, masks, counts = ref.plan(ctx, new, table, perm[at:], page, parents, words)
    cap = sum(new) + 7                                 # rows past the last token are padding
    wide = torch.full((len(ctx), width + 5), 77, dtype=torch.int32, device="cuda")
    block_table = wide[:, 2:2 + width]                 # a strided view: its surroundings stay as they are
    block_table.copy_(i32(table))
    par = None if parents is None else i32(np.concatenate([parents, np.full(7, -1)]))
    p = awq.paged_plan(i32(ctx), i32(new), block_table, i32(perm[at:]), page, cap, parents=par, mask_words=words)
    T = sum(new)
    assert p.cu_new.tolist() == cu and p.counts.tolist() == counts
    assert p.slot_map.tolist() == slots + [-1] * 7
    assert p.positions.tolist() == positions + [0] * 7
    assert p.token_request.tolist() == request + [-1] * 7
    assert np.array_equal(block_table.cpu().numpy(), want_table)
    assert (wide[:, :2] == 77).all() and (wide[:, 2 + width:] == 77).all()
    if words:
        got = p.tree_mask.cpu().numpy().view(np.uint32)
        assert np.array_equal(got[:T], masks) and not got[T:].any()


def test_plan_of_no_requests_and_of_deep_chains():
    p = awq.paged_plan(i32([]), i32([]), torch.empty((0, 4), dtype=torch.int32, device="cuda"), i32([]), 16, 3)
    assert p.cu_new.tolist() == [0] and p.counts.tolist() == [0, 0] and p.slot_map.tolist() == [-1] * 3
    n = 1000                                           # a chain given by its parents equals the chain without
    table = torch.full((1, 70), -1, dtype=torch.int32, device="cuda")
    free = i32(np.arange(70))
    a = awq.paged_plan(i32([0]), i32([n]), table.clone(), free, 16, n, parents=i32(np.arange(n) - 1), mask_words=32)
    b = awq.paged_plan(i32([0]), i32([n]), table.clone(), free, 16, n, mask_words=32)
    assert torch.equal(a.tree_mask, b.tree_mask) and torch.equal(a.positions, b.positions)


@pytest.mark.parametrize("requests", [6127, 6128, 6143, 6144, 16384])
def test_plan_of_many_requests(requests):
    """Two sums a request in shared memory, around the 48 KB that a kernel has without asking."""
    rng = np.random.default_rng(requests)
    ctx, new = rng.integers(0, 40, requests), rng.integers(0, 3, requests)
    have = -(-ctx // 16)
    need = int((-(-(ctx + new) // 16) - have).sum())
    perm = rng.permutation(int(have.sum()) + need)
    table = np.full((requests, 4), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = perm[at:at + n]
        at += n
    cu, want_table, slots, positions, request, _, counts = ref.plan(ctx.tolist(), new.tolist(), table, perm[at:], 16)
    buf = i32(table)
    p = awq.paged_plan(i32(ctx), i32(new), buf, i32(perm[at:]), 16, len(slots))
    assert p.cu_new.tolist() == cu and p.counts.tolist() == counts
    assert p.slot_map.tolist() == slots and p.positions.tolist() == positions and p.token_request.tolist() == request
    assert np.array_equal(buf.cpu().numpy(), want_table)


@pytest.mark.parametrize("what,status", [("free", Status.ERR_TOO_LARGE), ("width", Status.ERR_TOO_LARGE),
                                         ("tokens", Status.ERR_TOO_LARGE), ("mask", Status.ERR_TOO_LARGE),
                                         ("negative", Status.ERR_INVALID_ARG), ("parent", Status.ERR_INVALID_ARG),
                                         ("entry", Status.ERR_INVALID_ARG)])
def test_plan_reports_what_does_not_fit(what, status):
    """Exceeded capacities and bad entries give slot -1 or are ignored, and the device status says so."""
    ctx, new = [20, 3], [20, 14]                       # pages 2 + 1 of the first, 1 + 1 of the second
    table = np.array([[5, 6, -1, -1], [7, -1, -1, -1]])
    free = [1, 2]
    cap, words, parents = 34, 1, None
    if what == "free":
        free = [1]
    if what == "width":
        table = table[:, :2]
    if what == "tokens":
        cap = 30
    if what == "mask":
        ctx, new, free, cap = [0, 3], [40, 14], [1, 2, 3, 4], 54
        table[0] = -1
    if what == "negative":
        new = [20, -4]
    if what == "parent":
        parents = i32([-1] + [0] * 18 + [19] + [-1] * 14)   # node 19 its own parent
    if what == "entry":
        table[0, 1] = -3
    buf = i32(table)
    p = awq.paged_plan(i32(ctx), i32(new), buf, i32(free), 16, cap, parents=parents, mask_words=words)
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == status
    slots = p.slot_map.tolist()
    if what == "free":                                 # the second request finds none left
        assert slots[:20] == [6 * 16 + 4 + i for i in range(12)] + [16 + i for i in range(8)]
        assert slots[20:] == [7 * 16 + 3 + i for i in range(13)] + [-1] and p.counts.tolist() == [34, 2]
    if what == "width":
        assert slots[:20] == [6 * 16 + 4 + i for i in range(12)] + [-1] * 8
    if what == "tokens":
        assert p.cu_new.tolist() == [0, 20, 30] and p.counts.tolist() == [34, 2] and len(slots) == 30
    if what == "mask":
        assert (p.tree_mask[32:40] == -1).all()
    if what == "negative":
        assert p.cu_new.tolist() == [0, 20, 20] and slots[20:] == [-1] * 14
    if what == "parent":
        assert p.positions.tolist()[19] == 20 and p.tree_mask[19, 0].item() == 1 << 19
    if what == "entry":
        assert slots[:12] == [-1] * 12 and slots[12:20] == [16 + i for i in range(8)]


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("heads,dim,page", [(1, 8, 16), (8, 128, 16), (3, 40, 32), (32, 128, 64), (2, 256, 1024)])
@pytest.mark.parametrize("layout", ["token_major", "head_major"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_copies_into_slots(heads, dim, page, layout, dtype):
    gen = torch.Generator().manual_seed(heads * dim)
    T, blocks = 67, 9
    qkv = torch.randint(-2 ** 15, 2 ** 15, (T, 3 * heads, dim), dtype=torch.int16, generator=gen).cuda().view(dtype)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    slots = torch.randperm(blocks * page, generator=gen)[:T]
    slots[5] = -1
    slots[T - 1] = -1
    shape = (blocks, page, heads, dim) if layout == "token_major" else (blocks, heads, page, dim)
    ks, vs = (torch.full(shape, 3, dtype=torch.int16, device="cuda").view(dtype) for _ in range(2))
    kc, vc = (t if layout == "token_major" else t.transpose(1, 2) for t in (ks, vs))
    awq.kv_append(k, v, kc, vc, slots.cuda())
    for got, src in ((kc, k), (vc, v)):
        want = torch.full((blocks * page, heads, dim), 3, dtype=torch.int16)
        keep = slots >= 0
        want[slots[keep]] = src.view(torch.int16).cpu()[keep]
        assert torch.equal(got.reshape(blocks * page, heads, dim).view(torch.int16).cpu(), want)


def test_append_takes_what_the_kernel_before_has_just_written():
    """Back to back on one stream, an append reading the cache that the append before wrote:
    dependent launches, whose blocks may be on the GPU before those writes."""
    gen = torch.Generator().manual_seed(3)
    T, heads, dim = 512, 8, 128
    steps = [torch.randint(-2 ** 15, 2 ** 15, (T, heads, dim), dtype=torch.int16, generator=gen).cuda().view(torch.float16)
             for _ in range(8)]
    caches = torch.zeros((6, T // 16, 16, heads, dim), dtype=torch.float16, device="cuda")
    slots = torch.arange(T, device="cuda")
    for k in steps * 8:
        awq.kv_append(k, k, caches[0], caches[1], slots)
        for i in (2, 4):
            awq.kv_append(caches[i - 2].view(T, heads, dim), caches[i - 1].view(T, heads, dim), caches[i], caches[i + 1], slots)
    for cache in caches:
        assert torch.equal(cache.view(T, heads, dim).view(torch.int16), steps[-1].view(torch.int16))


def test_append_skips_and_reports_slots_outside_the_cache():
    k = torch.ones((3, 1, 8), dtype=torch.float16, device="cuda")
    cache = torch.zeros((2, 2, 16, 1, 8), dtype=torch.float16, device="cuda")
    awq.kv_append(k, k, cache[0], cache[1], torch.tensor([32, 3, -2], device="cuda"))
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    assert cache.sum().item() == 16 and (cache[:, 0, 3] == 1).all()


# ---------------------------------------------------------------- attention

class Step:
    """A random step: q, caches, table, lengths and a mask."""

    def __init__(self, ctx, new, heads, kv_heads, dim, page, dtype, mask, seed=0, garbage=float("nan")):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.ctx, self.new = list(ctx), list(new)
        self.cu = [0] + list(np.cumsum(new))
        self.T = self.cu[-1]
        self.table, blocks = tables(rng, ctx, new, page)
        self.q = torch.randn((self.T, heads, dim), generator=gen).to(dtype)
        self.k = torch.full((blocks, page, kv_heads, dim), garbage).to(dtype)
        self.v = self.k.clone()
        for b in range(len(ctx)):                      # only written slots hold numbers
            n = self.ctx[b] + self.new[b]
            at = torch.as_tensor(self.table[b][np.arange(n) // page]) * page + torch.arange(n) % page
            for cache in (self.k, self.v):
                cache.view(-1, kv_heads, dim)[at] = torch.randn((n, kv_heads, dim), generator=gen).to(dtype)
        self.words = -(-max(self.new) // 32)
        if mask == "causal":
            self.bits = None
        elif mask == "tree":
            par = forest(rng, new)
            self.bits = np.zeros((self.T, 32 * self.words), dtype=bool)
            for b in range(len(new)):
                for i in range(self.new[b]):
                    up = int(par[self.cu[b] + i])
                    if up >= 0:
                        self.bits[self.cu[b] + i] = self.bits[self.cu[b] + up]
                    self.bits[self.cu[b] + i, i] = True
        elif mask == "random":                         # any bits at all, later tokens and bits past the last one too
            self.bits = rng.random((self.T, 32 * self.words)) < 0.4
        elif mask == "none":                           # no drafted token is seen
            self.bits = np.zeros((self.T, 32 * self.words), dtype=bool)
        self.mask = None
        if self.bits is not None:
            packed = np.packbits(self.bits, axis=1, bitorder="little").view(np.int32)
            self.mask = torch.from_numpy(packed.copy())

    def run(self, scale=None, max_new=None, max_context=None, **kw):
        dim = self.q.shape[2]
        self.scale = dim ** -0.5 if scale is None else scale
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        out = awq.tree_attention(self.q.cuda(), self.k.cuda(), self.v.cuda(), i32(self.table), i32(self.ctx),
                                 i32(self.cu), self.scale, max(self.new) if max_new is None else max_new,
                                 max(self.ctx) if max_context is None else max_context,
                                 tree_mask=None if self.mask is None else self.mask.cuda(), lse=lse, **kw)
        return out, lse

    def check(self, out, lse, rows=slice(None)):
        want, want_lse, size = ref.attention(self.q, self.k, self.v, self.table, self.ctx, self.cu, self.scale, self.bits)
        u = U[self.q.dtype]
        got = out.double().cpu()
        bound = u * want.abs() + (u + 2.0 ** -13) * size + 2.0 ** -24
        err = (got - want).abs()
        assert (err <= bound)[rows].all(), f"worst {(err / bound)[rows].max().item():.3g} of the bound"
        gl, wl = lse.double().cpu()[rows], want_lse[rows]
        empty = wl == -torch.inf
        assert torch.equal(gl == -torch.inf, empty)
        assert ((gl - wl).abs()[~empty] <= 2.0 ** -13 * (1 + wl.abs()[~empty])).all()


HEADS = [(1, 1), (4, 4), (8, 1), (8, 2), (14, 2), (24, 1)]


@pytest.mark.parametrize("heads,kv_heads", HEADS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("mask", ["causal", "tree"])
def test_attention_heads_and_dims(heads, kv_heads, dim, dtype, mask):
    s = Step([130, 0, 17], [5, 3, 1], heads, kv_heads, dim, 16, dtype, mask, seed=heads + dim)
    s.check(*s.run())


@pytest.mark.parametrize("dim", [8, 40, 72, 80, 96, 136, 192, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attention_odd_head_dims(dim, dtype):
    for new in ([3, 2], [40, 9]):                      # few rows and many
        s = Step([70, 5], new, 4, 2, dim, 32, dtype, "tree", seed=dim)
        s.check(*s.run())


@pytest.mark.parametrize("ctx,new", [
    ([0], [1]), ([1], [1]), ([63], [1]), ([64], [1]), ([62], [2]), ([127], [1]), ([128], [1]), ([0], [64]),
    ([0, 0, 0], [1, 0, 2]), ([255, 256, 257], [1, 1, 1]), ([500], [33]), ([5], [129]), ([1000, 3], [17, 200]),
    ([3, 1000], [1, 7]), ([77] * 40, [1] * 40), ([0] * 20, [0] * 19 + [3])])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("mask", ["causal", "tree", "random"])
def test_attention_lengths(ctx, new, page, mask):
    s = Step(ctx, new, 8, 2, 64, page, torch.float16, mask, seed=sum(ctx) + page)
    s.check(*s.run())


@pytest.mark.parametrize("heads,kv_heads,new", [(8, 1, [1]), (2, 2, [1]), (8, 1, [9]), (8, 1, [40])])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_long_cache_is_split_and_joined(heads, kv_heads, new, dim):
    """One request whose keys are shared out over all CTAs, twice on the same scratch."""
    s = Step([20011], new, heads, kv_heads, dim, 32, torch.float16, "tree", seed=dim)
    out, lse = s.run()
    s.check(out, lse)
    again, lse2 = s.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)     # the order of the sums is fixed


@pytest.mark.parametrize("new", [[1, 1], [4, 30], [70, 3]])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attention_rows_that_see_nothing(new, dtype):
    """No context and an empty mask: zeros and -inf; beside it a request that has a context."""
    s = Step([0, 90], new, 4, 2, 64, 16, dtype, "none")
    out, lse = s.run()
    s.check(out, lse)
    assert (out[:new[0]] == 0).all() and (lse[:new[0]] == -torch.inf).all()


@pytest.mark.parametrize("new", [[6], [60]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attention_odd_values_in_unseen_keys_do_not_spread(new, bad, dtype):
    """A drafted token whose key and value are infinite or NaN: rows that do not see it are as if it were not there."""
    for where in ("k", "v"):
        s = Step([37], new, 8, 2, 128, 16, dtype, "tree", seed=new[0])
        node = new[0] // 2
        pos = 37 + node
        cache = getattr(s, where)
        cache[s.table[0][pos // 16], pos % 16, 0, 5] = bad
        out, lse = s.run()
        sees = s.bits[:s.T, node]
        assert sees.any() and not sees.all()
        s.check(out, lse, rows=torch.from_numpy(~sees))
        if where == "v":                               # and the others get it, in that element of that head only
            seen = out[torch.from_numpy(sees).cuda()].float()
            assert not seen[:, :4, 5].isfinite().any()
            seen[:, :4, 5] = 0
            assert seen.isfinite().all()


@pytest.mark.parametrize("new", [[2], [50]])
def test_attention_odd_values_in_the_context_reach_every_row(new):
    s = Step([37], new, 4, 2, 64, 16, torch.float16, "tree")
    s.v[s.table[0][0], 3, 1, 7] = float("nan")
    out, _ = s.run()
    assert out[:, 2:, 7].isnan().all()
    out[:, 2:, 7] = 0
    assert out.isfinite().all()


@pytest.mark.parametrize("new", [[3], [50]])
@pytest.mark.parametrize("scale", [0.0, 4.0, -0.3])
def test_attention_scales(new, scale):
    """Equal weights, weights all but one-hot, and a negative scale."""
    s = Step([150], new, 4, 1, 64, 16, torch.float16, "causal")
    s.check(*s.run(scale=scale))


@pytest.mark.parametrize("new", [[3, 1], [50, 20]])
def test_attention_strides(new):
    """q as a part of a fused projection's rows, heads before tokens in the cache, a strided table."""
    s = Step([45, 100], new, 8, 2, 64, 32, torch.bfloat16, "tree")
    s.scale = 0.125
    fused = torch.zeros((s.T, 14, 64), dtype=torch.bfloat16, device="cuda")
    fused[:, 3:11] = s.q.cuda()
    k = s.k.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    v = s.v.cuda().permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    wide = torch.full((2, 40), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + s.table.shape[1]] = i32(s.table)
    lse = torch.empty((s.T, 8), device="cuda")
    out = awq.tree_attention(fused[:, 3:11], k, v, wide[:, 3:3 + s.table.shape[1]], i32(s.ctx), i32(s.cu), 0.125,
                             max(new), 100, tree_mask=s.mask.cuda(), lse=lse)
    s.check(out, lse)


@pytest.mark.parametrize("new", [[2, 1], [2, 70]])
def test_attention_bounds_that_are_too_small_or_large(new):
    s = Step([300, 10], new, 8, 2, 64, 16, torch.float16, "tree")
    for bounds in ((0, 0), (1, 1), (500, 5000)):
        s.check(*s.run(max_new=bounds[0], max_context=bounds[1]))


def test_attention_with_bounds_of_any_size_has_the_whole_gpu():
    """The largest bounds that are taken: products of them that do not fit 64 bits left a CTA a head."""
    s = Step([600] * 256, [1] * 256, 64, 8, 64, 16, torch.float16, "causal", seed=2)
    args = (s.q.cuda(), s.k.cuda(), s.v.cuda(), i32(s.table), i32(s.ctx), i32(s.cu), 0.125)

    def ms(most):
        times = []
        for _ in range(6):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            out = awq.tree_attention(*args, most, most)
            end.record()
            end.synchronize()
            times.append(begin.elapsed_time(end))
        return min(times), out
    (tight, a), (loose, b) = ms(601), ms(2 ** 31 - 1)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -9
    assert loose <= 5 * tight


def test_attention_rows_past_the_last_token_stay():
    s = Step([30], [3], 4, 2, 64, 16, torch.float16, "causal")
    s.scale = 0.1
    q = torch.cat([s.q, torch.zeros(5, 4, 64, dtype=torch.float16)]).cuda()
    out = torch.full_like(q, 9.0)
    awq.tree_attention(q, s.k.cuda(), s.v.cuda(), i32(s.table), i32(s.ctx), i32(s.cu), 0.1, 3, 30, out=out)
    assert (out[3:] == 9).all() and (out[:3] != 9).all()


@pytest.mark.parametrize("what", ["cu_decreases", "cu_past_end", "ctx_negative", "ctx_past_table", "page"])
@pytest.mark.parametrize("new", [[2, 3], [40, 30]])
def test_attention_reports_bad_lengths_and_pages(what, new):
    s = Step([30, 40], new, 4, 2, 64, 16, torch.float16, "causal", garbage=0.0)
    ctx, cu, table = list(s.ctx), list(s.cu), s.table.copy()
    if what == "cu_decreases":
        cu[1] = cu[2] + 1
    if what == "cu_past_end":
        cu[2] += 1
    if what == "ctx_negative":
        ctx[0] = -1
    if what == "ctx_past_table":
        ctx[1] = 16 * table.shape[1]
    if what == "page":
        table[1, 0] = 10 ** 6
        table[0, 1] = -5
    out = torch.full((s.T, 4, 64), 5.0, dtype=torch.float16, device="cuda")
    awq.tree_attention(s.q.cuda(), s.k.cuda(), s.v.cuda(), i32(table), i32(ctx), i32(cu), 0.1, max(new), 40, out=out)
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    if what != "page":
        assert (out == 5).all()
    else:                                              # the pages read as zeros
        for b, pg in ((1, 0), (0, 1)):
            s.k[s.table[b, pg]] = 0
            s.v[s.table[b, pg]] = 0
        want, _, size = ref.attention(s.q, s.k, s.v, s.table, s.ctx, s.cu, 0.1, None)
        assert ((out.double().cpu() - want).abs() <= 2.0 ** -11 * want.abs() + (2.0 ** -11 + 2.0 ** -13) * size + 2.0 ** -24).all()


def test_attention_on_its_own_streams_at_once():
    steps = [Step([3000 + 64 * i], [n], 8, 2, 64, 16, torch.float16, "tree", seed=i)
             for i, n in enumerate([1, 5, 33, 2])]
    streams = [torch.cuda.Stream() for _ in steps]
    args = [(s.q.cuda(), s.k.cuda(), s.v.cuda(), i32(s.table), i32(s.ctx), i32(s.cu), s.mask.cuda()) for s in steps]
    torch.cuda.synchronize()
    outs = [[] for _ in steps]
    for _ in range(5):
        for s, st, a, o in zip(steps, streams, args, outs):
            with torch.cuda.stream(st):
                lse = torch.empty(s.q.shape[:2], device="cuda")
                o.append((awq.tree_attention(*a[:6], 0.125, max(s.new), max(s.ctx), tree_mask=a[6], lse=lse), lse))
    torch.cuda.synchronize()
    for s, o in zip(steps, outs):
        s.scale = 0.125
        s.check(*o[0])
        assert all(torch.equal(o[0][0], x) for x, _ in o[1:])


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^32 elements: its last blocks are read and written like its first."""
    page, heads, dim = 1024, 8, 128
    blocks = 2 ** 32 // (page * heads * dim) + 3
    k = torch.zeros((blocks, page, heads, dim), dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    gen = torch.Generator().manual_seed(3)
    new_k, new_v = (torch.randn((200, heads, dim), generator=gen).half().cuda() for _ in range(2))
    table = i32([[blocks - 1]])
    slots = (blocks - 1) * page + torch.arange(200, device="cuda")
    awq.kv_append(new_k, new_v, k, v, slots)
    for n in (1, 40):
        q = torch.randn((n, 8, dim), generator=gen).half()
        out = awq.tree_attention(q.cuda(), k, v, table, i32([200 - n]), i32([0, n]), 0.1, n, 200)
        want, _, size = ref.attention(q, new_k[None], new_v[None], np.array([[0]]), [200 - n], [0, n], 0.1)
        assert ((out.double().cpu() - want).abs() <= 2.0 ** -11 * want.abs() + (2.0 ** -11 + 2.0 ** -13) * size + 2.0 ** -24).all()


def test_attention_in_a_graph_follows_the_lengths():
    """Captured once on a reserved stream, replayed after the lengths have changed on the device."""
    first = Step([100, 7], [3, 2], 8, 2, 64, 16, torch.float16, "tree", seed=1)
    later = Step([333, 90], [2, 3], 8, 2, 64, 16, torch.float16, "tree", seed=2)
    stream = torch.cuda.Stream()
    assert awq.awq_reserve_tree_attention(64, stream.cuda_stream) == Status.OK
    with torch.cuda.stream(stream):
        width = later.table.shape[1]
        blocks = later.k.shape[0]
        q, mask = first.q.cuda(), first.mask.cuda()
        k = torch.zeros((blocks, 16, 2, 64), dtype=torch.float16, device="cuda")
        v = torch.zeros_like(k)
        k[:first.k.shape[0]], v[:first.v.shape[0]] = first.k.cuda(), first.v.cuda()
        table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
        table[:, :first.table.shape[1]] = i32(first.table)
        ctx, cu = i32(first.ctx), i32(first.cu)
        out, lse = torch.empty_like(q), torch.empty((5, 8), device="cuda")
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream, capture_error_mode="global"):
        awq.tree_attention(q, k, v, table, ctx, cu, 0.125, 3, 400, tree_mask=mask, out=out, lse=lse)
    first.scale = later.scale = 0.125
    graph.replay()
    torch.cuda.synchronize()
    first.check(out, lse)
    for dst, src in ((q, later.q), (k, later.k), (v, later.v), (mask, later.mask), (table, i32(later.table)),
                     (ctx, i32(later.ctx)), (cu, i32(later.cu))):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    later.check(out, lse)


# ---------------------------------------------------------------- attention, many rows
# Bounds that allow a long cache, or many row blocks, for which the tensor-core kernel is taken.
LONG = 2 ** 20


@pytest.mark.parametrize("heads,kv_heads", HEADS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("mask", ["causal", "tree"])
def test_many_rows_heads_and_dims(heads, kv_heads, dim, dtype, mask):
    s = Step([130, 0, 17], [35, 3, 1], heads, kv_heads, dim, 16, dtype, mask, seed=heads + dim)
    s.check(*s.run(max_context=LONG))


@pytest.mark.parametrize("dim", [8, 40, 72, 80, 96])
def test_many_rows_odd_head_dims(dim):
    for new in ([9, 2], [40, 9]):
        s = Step([70, 5], new, 4, 2, dim, 32, torch.float16, "tree", seed=dim)
        s.check(*s.run(max_context=LONG))


@pytest.mark.parametrize("ctx,new", [
    ([0], [64]), ([62], [5]), ([127], [9]), ([128], [33]), ([255, 256, 257], [5, 6, 7]), ([500], [33]), ([5], [129]),
    ([1000, 3], [17, 200]), ([3, 1000], [1, 7]), ([0] * 20, [0] * 19 + [9])])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("mask", ["causal", "tree", "random"])
def test_many_rows_lengths(ctx, new, page, mask):
    s = Step(ctx, new, 8, 2, 64, page, torch.float16, mask, seed=sum(ctx) + page)
    s.check(*s.run(max_context=LONG))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("mask", ["causal", "tree", "none"])
def test_many_rows_of_many_requests_with_short_caches(dim, dtype, mask):
    """Row blocks that are not cut, of 128 rows and of 256."""
    rng = np.random.default_rng(dim)
    for most in (24, 90):
        ctx, new = rng.integers(0, 300, 40), rng.integers(0, most + 1, 40)
        new[0], ctx[1] = most, 0
        s = Step(ctx, new, 8, 2, dim, 32, dtype, mask, seed=most)
        s.check(*s.run())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_rows_odd_values_in_unseen_keys_do_not_spread(bad, dtype):
    for where in ("k", "v"):
        s = Step([37], [60], 8, 2, 128, 16, dtype, "tree", seed=60)
        node = 30
        getattr(s, where)[s.table[0][(37 + node) // 16], (37 + node) % 16, 0, 5] = bad
        out, lse = s.run(max_context=LONG)
        sees = s.bits[:s.T, node]
        assert sees.any() and not sees.all()
        s.check(out, lse, rows=torch.from_numpy(~sees))
        if where == "v":
            seen = out[torch.from_numpy(sees).cuda()].float()
            assert not seen[:, :4, 5].isfinite().any()
            seen[:, :4, 5] = 0
            assert seen.isfinite().all()


@pytest.mark.parametrize("scale", [0.0, 4.0, -0.3])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_rows_scales_and_empty_rows(scale, dtype):
    s = Step([200, 0], [50, 20], 4, 2, 64, 16, dtype, "none", seed=5)
    out, lse = s.run(scale=scale, max_context=LONG)
    s.check(out, lse)
    assert (out[50:] == 0).all() and (lse[50:] == -torch.inf).all()


@pytest.mark.parametrize("ctx,heads,kv_heads", [([100], 32, 32), ([450], 8, 1), ([1000], 32, 8), ([1000] * 5, 16, 2),
                                                ([3900], 8, 8), ([7, 450, 0], 4, 2)])
@pytest.mark.parametrize("new", [1, 6])
@pytest.mark.parametrize("dim", [64, 96, 128, 200, 256])
def test_few_row_blocks_shared_by_clusters(ctx, heads, kv_heads, new, dim):
    s = Step(ctx, [new] * len(ctx), heads, kv_heads, dim, 32, torch.bfloat16, "tree", seed=dim + new)
    out, lse = s.run()
    s.check(out, lse)
    again, _ = s.run(max_new=max(1, new - 3))          # more row blocks than the bound allows for: several a cluster
    s.check(again, lse)


@pytest.mark.parametrize("rows", range(1, 17))
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (3, 1)])
def test_row_blocks_of_any_height_shared_by_clusters(rows, heads, kv_heads):
    """Lanes whose row a block does not have leave the join early and meet the others again."""
    new = -(-rows * kv_heads // heads)
    s = Step([500, 290], [new, 1], heads, kv_heads, 128, 16, torch.float16, "tree", seed=rows)
    for _ in range(20):
        out, lse = s.run()
    s.check(out, lse)


# ---------------------------------------------------------------- logits

class Rows:
    """Random logits with every control; `tree`: rows are the nodes of drafted trees."""

    def __init__(self, new, vocab, dtype, history=50, bias=5, grammar=True, seed=0):
        rng = np.random.default_rng(seed)
        self.B, self.R, self.V = len(new), sum(new), vocab
        self.x = torch.from_numpy(rng.normal(0, 3, (self.R, vocab)).astype(np.float32)).to(dtype)
        self.req = np.repeat(np.arange(self.B), new)
        self.hist = [list((vocab * rng.random(rng.integers(0, history + 1)) ** 2).astype(np.int64)) for _ in new]
        for h in self.hist[:1]:
            h += [-1, vocab - 1, 0, 0, 0]              # padding, the last token, a token said again
        self.prompt = [int(rng.integers(0, len(h) + 1)) for h in self.hist]
        self.rep = rng.uniform(0.8, 1.5, self.B).astype(np.float32)
        self.freq = rng.uniform(-0.3, 0.5, self.B).astype(np.float32)
        self.pres = rng.uniform(-0.3, 0.8, self.B).astype(np.float32)
        self.cu = [0] + list(np.cumsum(new))
        par = forest(rng, new)
        words = -(-max(list(new) + [1]) // 32)
        self.bits = np.zeros((self.R, 32 * words), dtype=bool)
        for b in range(self.B):
            for i in range(new[b]):
                up = int(par[self.cu[b] + i])
                if up >= 0:
                    self.bits[self.cu[b] + i] = self.bits[self.cu[b] + up]
                self.bits[self.cu[b] + i, i] = True
        self.draft = (vocab * rng.random(self.R) ** 2).astype(np.int64)
        self.path = [list(self.draft[self.cu[b] + np.nonzero(self.bits[r])[0]]) for r, b in enumerate(self.req)]
        self.bias = [sorted((int(t), float(np.float32(rng.normal()))) for t in rng.integers(0, vocab, bias))
                     for _ in new] if bias else None
        self.allowed = rng.random((self.R, vocab)) < 0.6 if grammar else None

    def arguments(self):
        kw = dict(row_request=i32(self.req), history=i32([t for h in self.hist for t in h]),
                  history_offsets=i32(np.cumsum([0] + [len(h) for h in self.hist])), prompt_lens=i32(self.prompt),
                  repetition=torch.from_numpy(self.rep).cuda(), frequency=torch.from_numpy(self.freq).cuda(),
                  presence=torch.from_numpy(self.pres).cuda(), draft_tokens=i32(self.draft), cu_new=i32(self.cu),
                  tree_mask=torch.from_numpy(np.packbits(self.bits, axis=1, bitorder="little").view(np.int32).copy()).cuda())
        if self.bias:
            kw.update(bias_tokens=i32([t for l in self.bias for t, _ in l]),
                      bias_values=torch.tensor([v for l in self.bias for _, v in l], dtype=torch.float32, device="cuda"),
                      bias_offsets=i32(np.cumsum([0] + [len(l) for l in self.bias])))
        if self.allowed is not None:
            pad = -self.V % 32
            kw["grammar_mask"] = torch.from_numpy(np.packbits(
                np.pad(self.allowed, ((0, 0), (0, pad))), axis=1, bitorder="little").view(np.int32).copy()).cuda()
        return kw

    def want(self):
        return ref.logits(self.x, self.req, self.B, self.hist, self.prompt, self.rep.astype(float),
                          self.freq.astype(float), self.pres.astype(float), self.path, self.bias, self.allowed)


def close(got, want, x):
    got = got.double().cpu().numpy()
    u = U[x.dtype]
    assert np.array_equal(got == -np.inf, want == -np.inf)
    fine = want != -np.inf
    bound = (u + 2.0 ** -21) * np.abs(want) + 2.0 ** -20 * (64 + np.abs(x.double().cpu().numpy())) + (2.0 ** -24 if u else 0)
    assert (np.abs(got[fine] - want[fine]) <= bound[fine]).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [1, 7, 8191, 8192, 8193, 32000, 50001])
@pytest.mark.parametrize("new", [[1], [3, 0, 5], [1, 40]])
def test_logits_all_controls(dtype, vocab, new):
    s = Rows(new, vocab, dtype, seed=vocab)
    x, kw = s.x.cuda(), s.arguments()
    got = awq.process_logits(x, **kw)
    close(got, s.want(), s.x)
    assert torch.equal(awq.process_logits(x, out=x, **kw), got)    # in place
    assert torch.equal(x, got)


@pytest.mark.parametrize("rows", [70, 1300])
def test_logits_many_rows_of_few_requests(rows):
    """Runs of rows that share a request's counts, and rows whose request changes back and forth."""
    s = Rows([rows // 2, rows - rows // 2], 999, torch.float32, history=300, seed=rows)
    close(awq.process_logits(s.x.cuda(), **s.arguments()), s.want(), s.x)
    s = Rows([1] * rows, 999, torch.float32, seed=rows)
    s.req = np.arange(rows) % 3
    s.path = None
    kw = s.arguments()
    for name in ("draft_tokens", "cu_new", "tree_mask"):
        kw.pop(name)
    close(awq.process_logits(s.x.cuda(), **kw), s.want(), s.x)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [600, 40001])
def test_logits_long_histories_and_many_biases(dtype, vocab):
    """Several batches of tokens, many or few of them in a range, and biases past those a thread keeps."""
    s = Rows([2, 1, 3], vocab, dtype, history=9000, bias=1300, seed=vocab)
    close(awq.process_logits(s.x.cuda(), **s.arguments()), s.want(), s.x)


def test_logits_rows_without_a_request():
    """The rows that a plan has past its tokens: as they are, and not reported."""
    s = Rows([2, 3], 5000, torch.bfloat16, grammar=False, seed=12)
    kw, x = s.arguments(), torch.cat([s.x, s.x[:2]]).cuda()
    for name, fill in (("row_request", -1), ("draft_tokens", 7), ("tree_mask", 1)):
        kw[name] = torch.cat([kw[name], torch.full_like(kw[name][:2], fill)])
    got = awq.process_logits(x, **kw)
    close(got[:5], s.want(), s.x)
    assert torch.equal(got[5:], x[5:])
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


@pytest.mark.parametrize("kinds", [(), ("rep",), ("freq",), ("pres",), ("bias",), ("grammar",), ("draft",)])
def test_logits_each_control_alone(kinds):
    s = Rows([2, 3], 9000, torch.float16, seed=4)
    kw, keep = s.arguments(), {"row_request", "history", "history_offsets", "prompt_lens"}
    keep |= {"rep": {"repetition"}, "freq": {"frequency"}, "pres": {"presence"}, "draft": {"draft_tokens", "cu_new", "tree_mask", "frequency"},
             "bias": {"bias_tokens", "bias_values", "bias_offsets"}, "grammar": {"grammar_mask"}}.get(kinds[0] if kinds else "", set())
    kw = {k: v for k, v in kw.items() if k in keep}
    one = lambda a, n: a.astype(float) if n in kw else None  # noqa: E731
    want = ref.logits(s.x, s.req, s.B, s.hist, s.prompt, one(s.rep, "repetition"), one(s.freq, "frequency"),
                      one(s.pres, "presence"), s.path if "draft_tokens" in kw else None,
                      s.bias if "bias_tokens" in kw else None, s.allowed if "grammar_mask" in kw else None)
    close(awq.process_logits(s.x.cuda(), **kw), want, s.x)
    if not kinds:
        assert torch.equal(awq.process_logits(s.x.cuda()), s.x.cuda())


def test_logits_chain_without_a_mask_rows_without_a_mask_and_strides():
    s = Rows([4, 2], 1001, torch.bfloat16, grammar=True, seed=8)
    kw = s.arguments()
    kw.pop("tree_mask")
    s.path = [list(s.draft[s.cu[b]:r + 1]) for r, b in enumerate(s.req)]
    kw["grammar_rows"] = i32([5, -1, 0, 0, -1, 2])
    s.allowed = np.stack([s.allowed[m] if m >= 0 else np.ones(1001, dtype=bool) for m in (5, -1, 0, 0, -1, 2)])
    wide = torch.zeros((6, 1200), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:1004] = s.x.cuda()
    close(awq.process_logits(wide[:, 3:1004], **kw), s.want(), s.x)
    out = torch.full((6, 1300), 3.0, dtype=torch.bfloat16, device="cuda")
    awq.process_logits(wide[:, 3:1004], out=out[:, 8:1009], **kw)
    close(out[:, 8:1009], s.want(), s.x)
    assert (out[:, :8] == 3).all() and (out[:, 1009:] == 3).all()


@pytest.mark.parametrize("rep", [1.1, 1.3, 3.0, 0.7, 1e-39, 1e38])
def test_logits_repetition_is_one_division(rep):
    """fp32 logits are divided, not multiplied by a rounded reciprocal: one rounding, and no overflow of the reciprocal."""
    x = torch.randn((2, 5000), generator=torch.Generator().manual_seed(1)) * 1e-3
    x[:, :40] = torch.tensor([2.0 ** e for e in range(-148, 128, 7)])
    x[:, 40:44] = torch.tensor([0.0, -0.0, float("inf"), -float("inf")])
    r = torch.tensor([rep, 1.7])
    got = awq.process_logits(x.cuda(), history=i32(np.tile(np.arange(5000), 2)), history_offsets=i32([0, 5000, 10000]),
                             repetition=r.cuda())
    x64, r64 = x.double(), r.double()[:, None]
    want = torch.where(x64 > 0, x64 / r64, x64 * r64).float()
    assert torch.equal(got.cpu(), want)


def test_logits_infinities_and_nan():
    x = torch.tensor([[float("inf"), -float("inf"), float("nan"), 1.0, float("nan"), 2.0]], device="cuda")
    got = awq.process_logits(x, history=i32([0, 1, 2, 3]), history_offsets=i32([0, 4]),
                             repetition=torch.tensor([2.0], device="cuda"),
                             grammar_mask=i32([[0b101111]])).tolist()[0]
    assert got[0] == float("inf") and got[1] == -float("inf") and got[2] != got[2]
    assert got[3] == 0.5 and got[4] == -float("inf") and got[5] == 2.0


@pytest.mark.parametrize("what", ["token", "request", "mask_row", "bias_order", "bias_token", "offset", "draft"])
def test_logits_reports_indices_out_of_range(what):
    s = Rows([2, 2], 500, torch.float32, seed=3)
    kw = s.arguments()
    if what == "token":
        kw["history"][3] = 500
    if what == "request":
        kw["row_request"][1] = 2
    if what == "mask_row":
        kw["grammar_rows"] = i32([0, 4, 1, 2])
    if what == "bias_order":
        kw["bias_tokens"][:2] = i32([9, 4])
    if what == "bias_token":
        kw["bias_tokens"][-1] = 2 ** 30
    if what == "offset":
        kw["history_offsets"][2] = 10 ** 9
    if what == "draft":
        kw["cu_new"][:] = i32([0, 4, 4])
    awq.process_logits(s.x.cuda(), **kw)
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
