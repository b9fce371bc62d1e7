"""GPU tests of rotary and rotary_append against references on the CPU.

Tolerance (u = 2^-11 for fp16, 2^-8 for bf16): one rounding to the type, u |ref| (and half of fp16's least
step, 2^-25); cosine and sine: their argument's rounding to fp32, pi 2^-25, and their own 2^-22, the two
products and their sum, 3 2^-24: together 2^-21 (|x_i| + |x_j|); the frequency in turns, 2^-52 of itself, which
the position multiplies: |position| inv_freq 2^-52 (|x_i| + |x_j|).
"""
import numpy as np
import pytest
import torch

import beam_reference as ref
import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import AWQError, Status

pytestmark = pytest.mark.gpu

FP16, BF16 = torch.float16, torch.bfloat16
U = {FP16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(autouse=True)
def _status(gpu):
    """Every test starts and ends with a clean device status."""
    awq.awq_last_device_status(None)
    yield
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


def i32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


def frequencies(n, base=10000.0):
    return (base ** -(torch.arange(n, dtype=torch.float64) / n)).float().cuda()


def check(got, x, positions, inv_freq, axes=None, pairs=False):
    p = positions.cpu().numpy().reshape(-1, x.shape[0])
    f = inv_freq.cpu().numpy()
    want, size = ref.rotary(x.double().cpu().numpy(), p, f, None if axes is None else axes.cpu().numpy(), pairs)
    far = np.abs(p.astype(np.float64)).max(initial=0) * float(f.max()) * 2.0 ** -52
    assert got.shape == x.shape and got.dtype == x.dtype
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= U[x.dtype] * np.abs(want) + (2.0 ** -21 + far) * size + 2.0 ** -25).all()
    n = 2 * len(f)
    assert torch.equal(got[..., n:], x[..., n:])


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,H,K,D,R", [
    (1, 1, 1, 8, 2), (1, 32, 32, 128, 128), (3, 8, 2, 64, 64), (7, 5, 1, 80, 32), (33, 4, 4, 72, 36), (5, 3, 3, 96, 20),
    (700, 2, 1, 128, 64), (1300, 1, 1, 16, 16), (65, 7, 1, 256, 256), (2, 2, 2, 1024, 1024), (9, 3, 1, 24, 24), (4, 200, 8, 64, 64)])
def test_rotary_matches_the_reference(dtype, pairs, T, H, K, D, R):
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    q = torch.randn((T, H, D), device="cuda", generator=gen).to(dtype)
    k = torch.randn((T, K, D), device="cuda", generator=gen).to(dtype)
    positions = torch.randint(0, 100000, (T,), device="cuda", generator=gen, dtype=torch.int32)
    f = frequencies(R // 2)
    before = q.clone(), k.clone()
    got_q, got_k = awq.rotary(q, k, positions, f, pairs=pairs)
    check(got_q, q, positions, f, pairs=pairs)
    check(got_k, k, positions, f, pairs=pairs)
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    only, none = awq.rotary(q, None, positions, f, pairs=pairs)
    assert none is None and torch.equal(only, got_q)
    # in place, as views of one projection's rows
    qkv = torch.cat([q, k, k], 1)
    view_q, view_k = qkv[:, :H], qkv[:, H:H + K]
    same_q, same_k = awq.rotary(view_q, view_k, positions, f, pairs=pairs, q_out=view_q, k_out=view_k)
    assert same_q is view_q and same_k is view_k
    assert torch.equal(view_q, got_q) and torch.equal(view_k, got_k) and torch.equal(qkv[:, H + K:], k)


@pytest.mark.parametrize("sections,interleaved", [((16, 24, 24), False), ((16, 24, 24), True), ((0, 1, 63), True), ((64,), False)])
@pytest.mark.parametrize("pairs", [False, True])
def test_several_axes(sections, interleaved, pairs):
    T = 301
    positions = torch.randint(-500, 500, (len(sections), T), device="cuda", dtype=torch.int32)
    axes = awq.rotary_axes(list(sections), interleaved)
    assert [(axes == a).sum().item() for a in range(len(sections))] == list(sections)
    q, k = torch.randn((T, 4, 128), device="cuda").half(), torch.randn((T, 2, 128), device="cuda").half()
    f = frequencies(64)
    got_q, got_k = awq.rotary(q, k, positions, f, axes=axes, pairs=pairs)
    check(got_q, q, positions, f, axes, pairs)
    check(got_k, k, positions, f, axes, pairs)


def test_axes_take_turns():
    assert awq.rotary_axes([2, 3, 1], interleaved=True).tolist() == [0, 1, 2, 0, 1, 1]
    assert awq.rotary_axes([2, 0, 3]).tolist() == [0, 0, 2, 2, 2]
    for bad in ([], [3, -1]):
        with pytest.raises(ValueError):
            awq.rotary_axes(bad)


def test_far_and_negative_positions():
    """Up to the ends of 32 bits, and frequencies above a turn a position."""
    positions = i32([2 ** 31 - 1, -2 ** 31, 16777217, -1, 0, 123456789])
    q = torch.randn((6, 2, 32), device="cuda").half()
    for f in (frequencies(16), torch.linspace(0.5, 20.0, 16, device="cuda"), -frequencies(16), torch.zeros(16, device="cuda")):
        got, _ = awq.rotary(q, None, positions, f)
        n = f.numel()
        want, size = ref.rotary(q.double().cpu().numpy(), positions.cpu().numpy()[None], f.cpu().numpy())
        # here per position and frequency
        far = np.abs(positions.cpu().numpy().astype(np.float64))[:, None] * np.abs(f.cpu().numpy()) * 2.0 ** -52
        far = np.concatenate([far, far], 1)[:, None]
        off = np.abs(got.double().cpu().numpy() - want)
        assert n == 16 and (off <= U[FP16] * np.abs(want) + (2.0 ** -21 + far) * size + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("T,H,K,D,R,page,heads_first", [
    (1, 32, 32, 128, 128, 16, False), (70, 8, 2, 64, 64, 16, True), (1000, 4, 4, 80, 32, 64, False), (5, 3, 1, 96, 20, 128, True)])
def test_append_is_rotary_and_append(dtype, T, H, K, D, R, page, heads_first):
    blocks = T // page + 4
    qkv = torch.randn((T, H + 2 * K, D), device="cuda").to(dtype)
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    positions, f = torch.randint(0, 9000, (T,), device="cuda", dtype=torch.int32), frequencies(R // 2)
    slots = torch.randperm(blocks * page, device="cuda")[:T]
    slots[::7] = -1
    make = lambda: torch.randn((blocks, K, page, D), device="cuda").to(dtype).transpose(1, 2) if heads_first \
        else torch.randn((blocks, page, K, D), device="cuda").to(dtype)  # noqa: E731
    caches = [make(), make()]
    before, want = [c.clone() for c in caches], [c.clone() for c in caches]
    want_q, want_k = awq.rotary(q, k, positions, f)
    awq.kv_append(want_k, v, *want, slots)
    got_q = awq.rotary_append(q, k, v, positions, f, *caches, slots)
    assert torch.equal(got_q, want_q)
    for got, w, b in zip(caches, want, before):
        assert torch.equal(got, w)
        untouched = torch.ones(blocks * page, dtype=torch.bool, device="cuda")
        untouched[slots[slots >= 0]] = False
        at = untouched.nonzero()[:, 0]
        assert torch.equal(got[at // page, at % page], b[at // page, at % page])
    q2 = q.clone()
    assert awq.rotary_append(q2, k, v, positions, f, *caches, slots, q_out=q2) is q2 and torch.equal(q2, want_q)


def test_bad_slots_and_axes_are_skipped_and_reported():
    q, k, f = torch.randn((3, 2, 64), device="cuda").half(), torch.randn((3, 2, 64), device="cuda").half(), frequencies(32)
    caches = [torch.zeros((2, 16, 2, 64), device="cuda", dtype=FP16) for _ in range(2)]
    slots = torch.tensor([32, 5, -2], device="cuda")
    got = awq.rotary_append(q, k, k, i32([1, 2, 3]), f, *caches, slots)
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    check(got, q, i32([1, 2, 3]), f)
    assert caches[1].flatten(0, 1).abs().sum((-1, -2)).nonzero().tolist() == [[5]]
    axes = torch.zeros(32, dtype=torch.int32, device="cuda")
    axes[3], axes[9] = 1, -1
    got, _ = awq.rotary(q, None, i32([1, 2, 3]), f, axes=axes)
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    f[3] = f[9] = 0
    check(got, q, i32([1, 2, 3]), f)


def test_no_tokens():
    q = torch.zeros((0, 4, 64), device="cuda", dtype=FP16)
    caches = [torch.zeros((2, 16, 4, 64), device="cuda", dtype=FP16) for _ in range(2)]
    a, b = awq.rotary(q, q, i32([]), frequencies(32))
    assert a.shape == b.shape == q.shape
    assert awq.rotary_append(q, q, q, i32([]), frequencies(32), *caches, torch.zeros(0, dtype=torch.int64, device="cuda")).shape == q.shape


def arguments():
    q, k = torch.zeros((3, 4, 64), device="cuda", dtype=FP16), torch.zeros((3, 2, 64), device="cuda", dtype=FP16)
    return dict(q=q, k=k, positions=i32([0, 1, 2]), inv_freq=frequencies(32), axes=torch.zeros(32, dtype=torch.int32, device="cuda"))


def append_arguments():
    cache = torch.zeros((2, 16, 2, 64), device="cuda", dtype=FP16)
    return dict(arguments(), v=torch.zeros((3, 2, 64), device="cuda", dtype=FP16), k_cache=cache, v_cache=cache.clone(),
                slot_map=torch.arange(3, device="cuda"))


@pytest.mark.parametrize("call,make", [(awq.rotary, arguments), (awq.rotary_append, append_arguments)])
def test_tensors_of_another_type_device_or_length(call, make):
    call(**make())
    for name, good in make().items():
        for bad in (good.cpu(), good.double(), good[:-1] if name != "k_cache" else good[:, :8]):
            with pytest.raises((ValueError, AWQError)):
                call(**dict(make(), **{name: bad}))
        with pytest.raises(TypeError):
            call(**dict(make(), **{name: 3}))


@pytest.mark.parametrize("name,bad", [
    ("q", lambda d: torch.zeros((3, 64, 4), device="cuda", dtype=FP16).transpose(1, 2)), ("k", lambda d: d["k"][..., :32]),
    ("inv_freq", lambda d: frequencies(33)), ("inv_freq", lambda d: frequencies(0)), ("positions", lambda d: d["positions"][None, None]),
    ("positions", lambda d: torch.zeros((0, 3), dtype=torch.int32, device="cuda")), ("q_out", lambda d: d["q"][:, :2]),
    ("k_out", lambda d: d["q"]), ("q_out", lambda d: d["q"].bfloat16())])
def test_shapes(name, bad):
    kw = arguments()
    kw[name] = bad(kw)
    with pytest.raises(ValueError):
        awq.rotary(**kw)


def test_statuses_of_the_library_become_its_error():
    with pytest.raises(AWQError, match="awq_rotary"):      # not on 16 bytes
        awq.rotary(torch.zeros(3 * 4 * 64 + 1, dtype=FP16, device="cuda")[1:].view(3, 4, 64), None, i32([0, 1, 2]), frequencies(32))
    q = torch.zeros((3, 4, 64), device="cuda", dtype=FP16)
    with pytest.raises(AWQError):                          # in place with other strides
        awq.rotary(q, None, i32([0, 1, 2]), frequencies(32), q_out=q.view(4, 3, 64).transpose(0, 1))
    with pytest.raises(AWQError):
        kw = append_arguments()
        kw.update(k_cache=torch.zeros((2, 24, 2, 64), device="cuda", dtype=FP16), v_cache=torch.zeros((2, 24, 2, 64), device="cuda", dtype=FP16))
        awq.rotary_append(**kw)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("R", [2, 6, 12, 14, 44, 60, 66, 128, 510, 1022])
def test_turned_parts_of_any_size(pairs, R):
    """Every width of a thread's item, heads of more items than a CTA has threads, into a cache."""
    D, T, H, K = (-(-R // 8) * 8 if R < 500 else 1024), 37, 3, 2
    qkv = torch.randn((T, H + 2 * K, D), device="cuda").half()
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    positions, f = torch.randint(0, 9000, (T,), device="cuda", dtype=torch.int32), frequencies(R // 2)
    caches = [torch.zeros((5, 16, K, D), device="cuda", dtype=FP16) for _ in range(2)]
    slots = torch.randperm(80, device="cuda")[:T]
    got_q, got_k = awq.rotary(q, k, positions, f, pairs=pairs)
    check(got_q, q, positions, f, pairs=pairs)
    check(got_k, k, positions, f, pairs=pairs)
    assert torch.equal(awq.rotary_append(q, k, v, positions, f, *caches, slots, pairs=pairs), got_q)
    assert torch.equal(caches[0].flatten(0, 1)[slots], got_k) and torch.equal(caches[1].flatten(0, 1)[slots], v)


@pytest.mark.parametrize("pairs,R", [(False, 4), (True, 4), (False, 8), (True, 2)])
def test_a_million_tokens_of_one_small_head(pairs, R):
    """A CTA has as many tokens as its shared memory holds angles of."""
    q = torch.randn((1_000_003, 1, 8), device="cuda").half()
    positions, f = torch.arange(1_000_003, device="cuda", dtype=torch.int32), frequencies(R // 2)
    check(awq.rotary(q, None, positions, f, pairs=pairs)[0], q, positions, f, pairs=pairs)
