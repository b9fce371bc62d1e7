"""GPU tests of beam_select's log-sum-exp: logits that a mask has made large and negative without making
them -inf, rows far from zero, and sums of which no part may be missing. Compared with 64 bits on the CPU.

Tolerance of a score, in units of 2^-24. An exponential 2^t is off by ln 2 |t| times what its argument is off by: at
most 2.5 of |t| (its roundings, and those of log2 e). Of n terms with weights 2^-|t| the mean |t| is below 7.5 for the 2048 of a
warp's part and below 10.5 for 2^14 parts: 2.5 ln 2 (7.5 + 10.5) = 31. The instruction: 4 for each of the two
exponentials. Additions of a lane 18, of the warp's lanes 5, of the single element 1, the parts' product 1, what the
rounding of the shift leaves 3. Together 67 of the sum, which is that much of its logarithm: taken as 100, whatever
the number of logits. The logarithm is good to 2^-28, and the score rounded to 2^-24 of itself.
"""
import numpy as np
import pytest
import torch

import beam_reference as ref
import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import Status

pytestmark = pytest.mark.gpu

FP16, BF16, FP32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _status(gpu):
    """Every test starts and ends with a clean device status."""
    awq.awq_last_device_status(None)
    yield
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


def tol(s):
    return 100 * 2.0 ** -24 + 2.0 ** -24 * abs(s)


def check_rows(logits, keep):
    """Every row a request of its own: its best tokens in order and their scores."""
    rows = logits.shape[0]
    before = -torch.arange(rows, device="cuda", dtype=torch.float32)[:, None] / 4
    step = awq.beam_select(logits, before, keep)
    live, _ = ref.beams(logits.double().cpu().numpy(), before.cpu().numpy(), keep)
    for b, want in enumerate(live):
        n = len(want)
        assert step.tokens[b].tolist() == [w[2] for w in want] + [-1] * (keep - n)
        assert step.parents[b].tolist() == [b] * n + [-1] * (keep - n)
        for got, w in zip(step.scores[b].tolist(), want):
            assert abs(got - w[0]) <= tol(w[0])


MASKS = [(d, -m) for d in (FP32, BF16) for m in (1e4, 1e5, 1e6, 1e8, 1e9, 1e10, 1e13, 1e16, 1e18, 1e20, 1e30, 1e36)] + \
        [(FP16, -1e4), (FP16, -6e4)]


@pytest.mark.parametrize("V", [9, 700, 50003])
@pytest.mark.parametrize("dtype,mask", MASKS)
def test_rows_with_finite_masks(dtype, mask, V):
    gen = torch.Generator(device="cuda").manual_seed(V)
    logits = torch.randn((6, V), device="cuda", generator=gen).mul_(3)
    logits[0, V // 5:V // 2] = mask                      # whole parts of the row
    logits[1, torch.rand(V, device="cuda", generator=gen) < 0.99] = mask
    logits[2, 5:] = mask                                 # fewer left than are kept: masked tokens come after them
    logits[3] = mask                                     # nothing but the mask
    logits[4, :V - 1] = mask
    logits[5, torch.arange(V, device="cuda") % 4096 > 7] = mask
    check_rows(logits.to(dtype), 9)


@pytest.mark.parametrize("V", [9, 700, 50003])
@pytest.mark.parametrize("dtype,offset", [(d, s * o) for d in (FP32, BF16) for s in (1, -1)
                                          for o in (4000, 4096, 4200, 1e4, 1e5, 1e6, 1e7, 1e20)] +
                         [(FP16, s * o) for s in (1, -1) for o in (4000, 4096, 4200, 1e4, 6e4)])
def test_rows_far_from_zero(dtype, offset, V):
    gen = torch.Generator(device="cuda").manual_seed(V)
    logits = torch.randn((4, V), device="cuda", generator=gen).mul_(3) + offset
    logits[1, ::2] = -offset                             # both at once
    logits[2] = offset
    check_rows(logits.to(dtype), 9)


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32])
@pytest.mark.parametrize("mask", [-1e4, -6e4])
def test_masked_beams_with_end_tokens(dtype, mask):
    """Several beams a request, each with tokens enough that its mask leaves."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn((12, 20011), device="cuda", generator=gen).mul_(3).to(dtype)
    logits[:, 4096:18000] = mask
    logits[::3, torch.rand(20011, device="cuda", generator=gen) < 0.9] = mask
    # scores so far apart that none are near one another
    before = torch.tensor([[-1.0, -400.0, -800.0, -1200.0]] * 3, device="cuda")
    ends = logits[0].float().topk(3).indices.int()
    step = awq.beam_select(logits, before, 7, end_tokens=ends)
    live, ended = ref.beams(logits.double().cpu().numpy(), before.cpu().numpy(), 7, set(ends.tolist()))
    for want_all, s, p, t in ((live, *step[:3]), (ended, *step[3:])):
        for b, want in enumerate(want_all):
            n = len(want)
            assert list(zip(p[b].tolist(), t[b].tolist())) == [w[1:] for w in want] + [(-1, -1)] * (7 - n)
            assert all(abs(g - w[0]) <= tol(w[0]) for g, w in zip(s[b].tolist(), want))


@pytest.mark.parametrize("dtype", [FP16, FP32])
@pytest.mark.parametrize("V", [2 ** 20, 2 ** 22 + 5, 2 ** 24 + 3])
def test_no_part_of_a_long_row_is_missing(dtype, V):
    """A warp's part of 4 KB is 2^-13 of the longest of these sums, 2^11 times what the tolerance allows."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    check_rows(torch.randn((1, V), device="cuda", generator=gen).to(dtype), 32)


@pytest.mark.parametrize("R,W,V,keep,dtype", [(125, 2, 70000, 8, BF16), (5, 3, 290000, 16, FP32), (143, 7, 50001, 4, BF16),
                                              (44, 32, 33377, 32, FP16), (77, 8, 70003, 8, BF16), (1, 2, 1_100_000, 32, FP32)])
def test_sums_however_rows_are_shared_out(R, W, V, keep, dtype):
    gen = torch.Generator(device="cuda").manual_seed(R + V)
    logits = torch.randn((R * W, V), generator=gen, device="cuda").to(dtype)
    before = -torch.rand((R, W), generator=gen, device="cuda")
    step = awq.beam_select(logits, before, keep)
    at = step.parents.long().flatten(), step.tokens.long().flatten()
    want = before.double().flatten()[at[0]] + logits.double()[at] - torch.stack(
        [row.double().logsumexp(0) for row in logits])[at[0]]
    assert ((step.scores.double().flatten() - want).abs() <= tol(want)).all()


@pytest.mark.parametrize("V", [2, 3, 5, 6, 7, 11, 23, 47, 85, 86, 171, 341, 342, 1000, 1365, 1366, 2731, 5461, 10007, 21845,
                               50257, 87381, 87382, 131071, 151936, 349525, 699051, 1048575, 1398102, 2097151])
def test_the_logarithm(V):
    """Equal logits: their sum is a whole number, exact in fp32, and a score next to ln V cancels all but what
    the logarithm is off by. Its series behind the first term (0.0056 at most) is in fp32: four roundings of the terms and three
    of additions, 2^-24 of it each, below 2^-28."""
    before = np.float32(np.log(V))
    step = awq.beam_select(torch.zeros((1, V), device="cuda"), torch.tensor([[float(before)]], device="cuda"), 1)
    want = float(np.longdouble(before) - np.log(np.longdouble(V)))
    assert abs(step.scores.item() - want) <= 2.0 ** -28 + 2.0 ** -24 * abs(want)
