"""GPU tests of beam_select and reorder_states against 64-bit references on the CPU.

Tolerance of a score: the log-sum-exp's fp32 parts. Each exponential is off by 2^-22 of its value
(the instruction) and by 2^-24 |t| / 2^|t| of the row's largest (its argument t's rounding), below 2^-24;
a thread adds its `n` terms one by one, 2^-24 of the sum each, then 16 sums are joined: together
(n + 32) 2^-24 of the sum, which is that much of its logarithm. The score is rounded once more: 2^-24 of
its value. Parents and tokens are the reference's wherever scores of different rows are further apart than
that; within a row the order is the logits' own, without any tolerance.
"""
import numpy as np
import pytest
import torch

import beam_reference as ref
import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import AWQError, Status

pytestmark = pytest.mark.gpu

FP16, BF16, FP32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _status(gpu):
    """Every test starts and ends with a clean device status."""
    awq.awq_last_device_status(None)
    yield
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


def i32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


def check(logits, before, keep, ends=()):
    """Runs beam_select and compares it with the reference; returns what it gave."""
    B, W = before.shape
    V = logits.shape[1]
    step = awq.beam_select(logits, before, keep, end_tokens=i32(list(ends)) if ends else None)
    x = logits.double().cpu().numpy()
    live, ended = ref.beams(x, before.cpu().numpy(), keep, set(ends))
    every = ref.scores(x, before.cpu().numpy()).reshape(B * W, V)
    tol = lambda s: (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -24 * abs(s)  # noqa: E731
    for want_all, names in ((live, ("scores", "parents", "tokens")),
                            (ended, ("ended_scores", "ended_parents", "ended_tokens"))):
        if names[0] == "ended_scores" and not ends:
            assert step.ended_scores is None and step.ended_parents is None and step.ended_tokens is None
            continue
        s, p, t = (getattr(step, n).cpu().numpy() for n in names)
        assert s.shape == p.shape == t.shape == (B, keep) and s.dtype == np.float32
        for b, want in enumerate(want_all):
            n = len(want)
            got = list(zip(s[b, :n].tolist(), p[b, :n].tolist(), t[b, :n].tolist()))
            # near scores of different rows may change places, and then come in or fall out at the end
            every_b = live[b] + ended[b]
            near = any(abs(a[0] - c[0]) <= 4 * tol(a[0]) and a[1] != c[1] for a in every_b for c in every_b)
            flat = np.sort(every[b * W:(b + 1) * W][np.isfinite(every[b * W:(b + 1) * W])])[::-1]
            k = len(every_b)
            near = near or (W > 1 and 0 < k < len(flat) and flat[k - 1] - flat[k] <= 4 * tol(flat[k]))
            if not near:
                assert [g[1:] for g in got] == [w[1:] for w in want]
                assert (s[b, n:] == -np.inf).all() and (p[b, n:] == -1).all() and (t[b, n:] == -1).all()
            for (gs, gp, gt), w in zip(got, want):
                if gp < 0:
                    assert near
                    continue
                assert abs(gs - w[0]) <= tol(w[0])
                assert abs(every[gp, gt] - gs) <= tol(gs)
            assert len({g[1:] for g in got if g[1] >= 0}) == len([g for g in got if g[1] >= 0])
            for row in {g[1] for g in got if g[1] >= 0}:       # the order within a row
                mine = [g[2] for g in got if g[1] == row]
                assert mine == sorted(mine, key=lambda v: (-(x[row, v] + 0.0), v))
    return step


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32])
@pytest.mark.parametrize("B,W,V,keep,ends", [
    (1, 1, 1, 1, 0), (1, 1, 7, 4, 0), (1, 4, 32000, 4, 1), (3, 5, 1000, 5, 3), (2, 32, 2049, 32, 8), (1, 1, 50257, 8, 2),
    (5, 8, 10007, 3, 1), (2, 3, 100003, 7, 2), (40, 2, 333, 2, 1), (1, 32, 4096, 1, 0), (1, 2, 700001, 16, 8)])
def test_beams_match_the_reference(dtype, B, W, V, keep, ends):
    gen = torch.Generator(device="cuda").manual_seed(V + keep)
    logits = torch.randn((B * W, V), device="cuda", generator=gen).mul_(3).to(dtype)
    before = -10 - 2 * torch.rand((B, W), device="cuda", generator=gen)
    # end tokens that matter: some rows' best
    stops = sorted({int(t) for t in logits.float().argmax(-1)[:ends].tolist()} | set(range(0, min(ends, V))))[:ends]
    check(logits, before, keep, stops)


@pytest.mark.parametrize("dtype", [FP16, FP32])
@pytest.mark.parametrize("kind", ["equal", "few", "descending", "ascending", "periodic", "one_place", "zeros"])
def test_ties_and_orders(dtype, kind):
    """Equal logits go by the lowest token; data whose best lie together are found as well."""
    B, W, V, keep = 2, 3, 20011, 9
    gen = torch.Generator(device="cuda").manual_seed(5)
    at = torch.arange(V, device="cuda")
    logits = {"equal": torch.full((V,), 1.5, device="cuda"), "descending": -at / 64.0, "ascending": at / 64.0 % 200.0,
              "few": torch.randint(3, (V,), device="cuda", generator=gen).float(),
              # the best all at one residue of the pieces that a thread reads
              "periodic": (at % 2048 < 8).float() * (10 + at / V),
              # and all of them with one thread
              "one_place": (at % 8192 < 64).float() * (10 + at / V),
              "zeros": torch.where(at % 2 == 0, -0.0, 0.0)}[kind]
    logits = logits.expand(B * W, V).to(dtype).contiguous()
    # rows far apart, so that rows do not tie
    before = torch.tensor([[-1.0, -2.25, -4.5], [-7.0, -3.0, -5.125]], device="cuda")
    check(logits, before, keep, (1, 4))


def test_equal_scores_go_by_the_lower_row():
    logits = torch.randn((4, 5000), device="cuda").half()
    logits[1:] = logits[:1]
    step = awq.beam_select(logits, torch.full((1, 4), -3.0, device="cuda"), 10)
    # tokens of one fp16 logit tie too: score, row, token
    top = logits[0].float().sort(descending=True)
    want = sorted((-x, r, t) for x, t in zip(top.values[:20].tolist(), top.indices[:20].tolist()) for r in range(4))[:10]
    assert step.tokens[0].tolist() == [t for _, _, t in want]
    assert step.parents[0].tolist() == [r for _, r, _ in want]


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32])
def test_masked_rows_and_dead_beams(dtype):
    """-inf is no candidate, the type's lowest value is one; beams of -inf are not looked at."""
    lowest = torch.finfo(dtype).min
    gen = torch.Generator(device="cuda").manual_seed(9)
    logits = torch.randn((12, 3001), device="cuda", generator=gen).to(dtype)
    logits[0] = -torch.inf                       # a row that its mask leaves nothing
    logits[1, 5:] = -torch.inf
    logits[2] = lowest
    logits[3, 7:] = lowest
    logits[4] = -torch.inf
    logits[4, 3000] = lowest
    logits[5, torch.rand(3001, device="cuda", generator=gen) < 0.99] = -torch.inf
    logits[6] = torch.nan                        # not looked at
    logits[7, 9] = torch.inf
    before = -torch.rand((3, 4), device="cuda", generator=gen)
    before[1, 2:] = -torch.inf
    check(logits, before, 6, (2,))
    before[2] = -torch.inf                       # no beam at all
    step = check(logits, before, 6, (2,))
    assert (step.parents[2] == -1).all() and (step.ended_parents[2] == -1).all()


@pytest.mark.parametrize("V", [500, 300000])
def test_scores_below_the_least_fp32_number(V):
    """They are rounded to -inf, and their tokens are candidates all the same."""
    logits = torch.full((2, V), torch.finfo(FP32).min, device="cuda")
    logits[:, 7] = 3e38
    logits[1, 9:] = -torch.inf
    step = awq.beam_select(logits, torch.tensor([[-1.0], [-2.0]], device="cuda"), 4)
    assert step.tokens[0].tolist() == [7, 0, 1, 2] and step.tokens[1].tolist() == [7, 0, 1, 2]
    assert step.parents.tolist() == [[0] * 4, [1] * 4] and step.scores.tolist() == [[-1.0] + [-torch.inf] * 3, [-2.0] + [-torch.inf] * 3]


@pytest.mark.parametrize("requests", [1, 3, 38, 39])
@pytest.mark.parametrize("V", [9, 8191, 8192, 20000])
def test_few_and_many_requests_give_the_same(requests, V):
    """However the rows are shared out over CTAs."""
    logits = torch.randn((39 * 3, V), device="cuda").half()
    before = -torch.rand((39, 3), device="cuda")
    before[2, 1] = -torch.inf
    every = awq.beam_select(logits, before, 7, end_tokens=i32([3, 5]))
    some = awq.beam_select(logits[:3 * requests], before[:requests], 7, end_tokens=i32([3, 5]))
    for a, b in zip(some, every):
        assert torch.equal(a, b[:requests])


@pytest.mark.parametrize("bad", [torch.nan, torch.inf])
@pytest.mark.parametrize("where", [0, 4999, 10002])
def test_rows_with_nan_or_infinity_have_no_candidates_and_are_reported(bad, where):
    logits = torch.randn((4, 10003), device="cuda").bfloat16()
    logits[1, where] = bad
    step = awq.beam_select(logits, torch.zeros((1, 4), device="cuda"), 8)
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    assert set(step.parents[0].tolist()) <= {0, 2, 3} and (step.tokens >= 0).all()
    before = torch.tensor([[0.0, bad, 0.0, 0.0]], device="cuda")
    step = awq.beam_select(torch.randn((4, 100), device="cuda"), before, 8)
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    assert set(step.parents[0].tolist()) <= {0, 2, 3}


@pytest.mark.parametrize("dtype", [FP16, FP32])
@pytest.mark.parametrize("offset", [0, 1, 3, 7])
def test_rows_at_any_element(dtype, offset):
    wide = torch.full((6, 4100), torch.nan, device="cuda", dtype=dtype)       # what lies between the rows does not matter
    logits = wide[:, offset:offset + 4001]
    logits.copy_(torch.randn((6, 4001), device="cuda"))
    check(logits, -torch.rand((2, 3), device="cuda"), 5, (17,))


def test_end_tokens():
    """A candidate that ends counts among the first num_beams of all, and takes no place of those that go on."""
    logits = torch.full((2, 50), -5.0, device="cuda")
    logits[0, [3, 4, 9]] = torch.tensor([4.0, 3.0, 2.0], device="cuda")
    logits[1, [4, 8]] = torch.tensor([3.5, 1.0], device="cuda")
    step = check(logits, torch.tensor([[0.0, -0.5]], device="cuda"), 2, (3, 4, 4, 99, -1))
    assert step.tokens[0].tolist() == [9, 8] and step.parents[0].tolist() == [0, 1]
    assert step.ended_tokens[0].tolist()[0] == 3 and step.ended_parents[0].tolist()[1] in (0, 1)
    # all that there is ends
    step = awq.beam_select(torch.zeros((1, 3), device="cuda"), torch.zeros((1, 1), device="cuda"), 2, end_tokens=i32([0, 1, 2]))
    assert (step.parents == -1).all() and step.ended_tokens[0].tolist() == [0, 1]


def test_an_empty_list_of_end_tokens():
    step = awq.beam_select(torch.randn((3, 50), device="cuda"), torch.zeros((1, 3), device="cuda"), 4, end_tokens=i32([]))
    assert (step.ended_scores == -torch.inf).all() and (step.ended_parents == -1).all() and (step.ended_tokens == -1).all()


def test_a_row_gives_the_same_alone_and_among_others():
    """Bit for bit, wherever it lies in the batch and however the batch is shared out."""
    for V in (32000, 151936):
        logits = torch.randn((60, V), device="cuda").bfloat16()
        before = -torch.rand((60, 1), device="cuda")
        every = awq.beam_select(logits, before, 5)
        for r in (0, 7, 59):
            one = awq.beam_select(logits[r:r + 1], before[r:r + 1], 5)
            assert torch.equal(one.scores[0], every.scores[r]) and torch.equal(one.tokens[0], every.tokens[r])


def test_no_requests():
    step = awq.beam_select(torch.zeros((0, 10), device="cuda"), torch.zeros((0, 4), device="cuda"), 4, end_tokens=i32([1]))
    assert step.scores.shape == (0, 4) and step.ended_tokens.shape == (0, 4)


@pytest.mark.parametrize("V", [2 ** 22 + 5, 2 ** 24 + 3])
def test_a_large_vocabulary_is_read_in_several_rounds(V):
    at = torch.arange(V, device="cuda")
    # among others the best with few threads, or one, so that lists fill up
    for row in ((at % 2048 < 8).half() * (at / V).half(), (at % 8192 < 64).half() * (at / V).half(),
                torch.randn(V, device="cuda").half()):
        check(row[None], torch.zeros((1, 1), device="cuda"), 32, (7,))


# ---------------------------------------------------------------- states

@pytest.mark.parametrize("dtype", [torch.uint8, torch.bool, FP16, torch.int32, torch.int64, torch.complex128])
@pytest.mark.parametrize("shape", [(), (1,), (3,), (7, 5), (1000,), (4099,), (0,), (2, 1, 8)])
def test_states_follow_their_parents(dtype, shape):
    gen = torch.Generator().manual_seed(3)
    a = torch.randint(0, 2 if dtype == torch.bool else 100, (9, *shape), generator=gen).to(dtype).cuda()
    parents = i32([3, 3, 0, 8, -1, 5, 2, 2, 2, 7, 1])
    got, = awq.reorder_states([a], parents)
    want = a[parents.clamp(min=0).long()]
    want[4] = 0
    assert got.dtype == dtype and torch.equal(got, want)


def test_states_with_strides_and_outputs():
    a, b = torch.arange(40 * 12, device="cuda").view(40, 12).short(), torch.randn((40, 3, 64), device="cuda")
    parents = torch.randint(-1, 40, (25,), device="cuda", dtype=torch.int32)
    outs = [torch.full((25, 9), -7, device="cuda", dtype=torch.int16)[:, 1:8], torch.empty((25, 3, 64), device="cuda")]
    made = awq.reorder_states([a[:, 3:10], b], parents, outs=outs)
    keep = (parents >= 0)[:, None]
    assert made[0].data_ptr() == outs[0].data_ptr() and made[1].data_ptr() == outs[1].data_ptr()
    assert torch.equal(outs[0], torch.where(keep, a[:, 3:10][parents.clamp(min=0).long()], 0))
    assert torch.equal(outs[1], torch.where(keep[..., None], b[parents.clamp(min=0).long()], 0.0))


def test_many_states_and_none():
    states = [torch.randn((5, 1 + i), device="cuda") for i in range(150)]
    parents = i32([4, 0, 0])
    for s, got in zip(states, awq.reorder_states(states, parents)):
        assert torch.equal(got, s[parents.long()])
    assert awq.reorder_states([], parents) == []
    got, = awq.reorder_states([states[3]], i32([]))
    assert got.shape == (0, 4)
    got, = awq.reorder_states([torch.zeros((0, 6), device="cuda")], i32([-1, -1]))
    assert got.shape == (2, 6) and (got == 0).all()


def test_bad_parents_give_zeros_and_are_reported():
    a = torch.ones((4, 10), device="cuda")
    got, = awq.reorder_states([a], i32([0, 4, -2, 3]))
    assert got.sum(-1).tolist() == [10, 0, 0, 10]
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG


# ---------------------------------------------------------------- refusals

@pytest.mark.parametrize("change", [
    dict(logits=lambda d: d["logits"].cpu()), dict(logits=lambda d: d["logits"].double()),
    dict(logits=lambda d: torch.zeros((100, 8), device="cuda").T), dict(logits=lambda d: d["logits"][:7]),
    dict(logits=lambda d: d["logits"][:, :0]), dict(scores=lambda d: d["scores"].half()),
    dict(scores=lambda d: d["scores"].view(-1)), dict(scores=lambda d: d["scores"].T), dict(scores=lambda d: torch.zeros((8, 0), device="cuda")),
    dict(num_beams=lambda d: 0), dict(num_beams=lambda d: 33), dict(end_tokens=lambda d: i32(range(9))),
    dict(end_tokens=lambda d: torch.zeros(2, device="cuda")), dict(end_tokens=lambda d: torch.zeros(2, dtype=torch.int32)),
    dict(scores=lambda d: torch.zeros((0, 33), device="cuda"), logits=lambda d: d["logits"][:0])])
def test_beam_select_refuses(change):
    kw = dict(logits=torch.zeros((8, 100), device="cuda"), scores=torch.zeros((2, 4), device="cuda"), num_beams=4,
              end_tokens=i32([1]))
    awq.beam_select(**kw)
    kw.update({k: f(kw) for k, f in change.items()})
    with pytest.raises(ValueError):
        awq.beam_select(**kw)
    with pytest.raises(TypeError):
        awq.beam_select(None, kw["scores"], 4)


def test_reorder_states_refuses():
    a, parents = torch.zeros((4, 10), device="cuda"), i32([0, 1])
    for states, p, outs in [([a.cpu()], parents, None), ([a], parents.cpu(), None), ([a], parents.long(), None),
                            ([a], parents[None], None), ([a.T], parents, None), ([a, a[:3]], parents, None),
                            ([torch.zeros((), device="cuda")], parents, None), ([a], parents, []),
                            ([a], parents, [torch.zeros((3, 10), device="cuda")]),
                            ([a], parents, [torch.zeros((2, 11), device="cuda")]),
                            ([a], parents, [torch.zeros((2, 10), device="cuda", dtype=FP16)]),
                            ([a], parents, [a[1:3]]), ([a], parents, [torch.zeros((10, 2), device="cuda").T])]:
        with pytest.raises(ValueError):
            awq.reorder_states(states, p, outs=outs)
    for states in (a, None, [1], 5):
        if states is not a:
            with pytest.raises(TypeError):
                awq.reorder_states(states, parents)
    assert issubclass(AWQError, RuntimeError)


@pytest.mark.parametrize("R,W,V,keep,ends,dtype", [
    (125, 2, 70000, 8, 0, BF16),      # two parts of each row, some with a chunk fewer
    (5, 3, 290000, 16, 3, FP32),      # a chunk a part
    (143, 7, 50001, 4, 1, BF16),      # two rows a part, the last part of one
    (44, 32, 33377, 32, 8, FP16),     # a row a part, more parts than CTAs at once
    (77, 8, 70003, 8, 0, BF16),       # parts that end within rows
    (1, 2, 1_100_000, 32, 8, FP32),   # parts of many chunks
    (1, 32, 1_600_000, 32, 8, BF16),  # of more than have their maxima kept
])
def test_ways_to_share_out_the_rows(R, W, V, keep, ends, dtype):
    gen = torch.Generator(device="cuda").manual_seed(R + V)
    logits = torch.randn((R * W, V), generator=gen, device="cuda").to(dtype)
    scores = -torch.rand((R, W), generator=gen, device="cuda")
    end_tokens = torch.randperm(V, generator=gen, device="cuda")[:ends].int() if ends else None
    step = awq.beam_select(logits, scores, keep, end_tokens)
    x = logits.double()
    s = (scores.double().reshape(-1, 1) + torch.log_softmax(x, 1)).reshape(R, W * V)
    if ends:
        s[:, (torch.arange(W, device="cuda")[:, None] * V + end_tokens[None]).flatten()] = -torch.inf
    want = s.topk(keep).values
    bound = (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -24 * want.abs()        # of sums and scores, as in check
    assert ((step.scores.double() - want).abs() <= bound).all()
    at = step.parents.long() % W * V + step.tokens.long()
    assert (torch.div(step.parents, W, rounding_mode="floor") == torch.arange(R, device="cuda")[:, None]).all()
    assert ((s.gather(1, at) - want).abs() <= 2 * bound).all() and all(len(set(a)) == keep for a in at.tolist())
