"""The tensor-core kernel of tree_attention, taken because the bounds allow a long cache,
in the forms in which it differs from the few-row kernel: its own products, tensor maps
and pieces. Tolerances as in test_gpu_step.py."""
import numpy as np
import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
import step_reference as ref
from bit_weight_quantized_awq_gb300 import Status
from test_gpu_step import LONG, Step, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status(gpu):
    """Every test starts and ends with a clean device status."""
    awq.awq_last_device_status(None)
    yield
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


@pytest.fixture(scope="module", autouse=True)
def _profiler(gpu):
    """The first session of a process may miss kernels while the tracing library starts up."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]):
        torch.ones(1024, device="cuda").sum()
        torch.cuda.synchronize()


def kernels_of(call):
    """Names of the library's kernels that `call` launches; none if the profiler records none here."""
    torch.cuda.synchronize()
    activities = [torch.profiler.ProfilerActivity.CPU, torch.profiler.ProfilerActivity.CUDA]
    with torch.profiler.profile(activities=activities) as prof:
        call()
        torch.cuda.synchronize()
    return [e.name for e in prof.events()
            if e.device_type == torch.autograd.DeviceType.CUDA and "attention" in e.name and "awq" in e.name]


def on_tensor_cores(call, joined=None):
    """`call` takes the tensor-core kernel, and with a join or without one if that is given."""
    names = kernels_of(call)
    if not names:
        return
    assert any("attention_tc_kernel" in n for n in names) and not any("attention_rows_kernel" in n for n in names), names
    if joined is not None:
        assert any("attention_join_kernel" in n for n in names) == joined, names


def close(out, want, size, u=2.0 ** -11):
    err = (out.double().cpu() - want).abs()
    assert (err <= u * want.abs() + (u + 2.0 ** -13) * size + 2.0 ** -24).all()


@pytest.mark.parametrize("heads,kv_heads,new", [(8, 8, 26), (16, 2, 13), (16, 2, 64)])
@pytest.mark.parametrize("dim", [64, 128])
def test_every_call_gives_the_same_bits(heads, kv_heads, new, dim):
    """S of a tile is written over the weights of the tile before: only after their product
    with V. Streams, halves and CTAs meet in another order from call to call; the sums do not."""
    s = Step([3000, 700, 1500, 90], [new, new // 2, new, 1], heads, kv_heads, dim, 32, torch.float16, "tree", seed=new)
    out, lse = s.run(max_context=LONG)
    s.check(out, lse)
    args = (s.q.cuda(), s.k.cuda(), s.v.cuda(), i32(s.table), i32(s.ctx), i32(s.cu))
    mask = s.mask.cuda()
    for _ in range(200):
        assert torch.equal(awq.tree_attention(*args, s.scale, new, LONG, tree_mask=mask), out)


@pytest.mark.parametrize("kv_heads", [1, 8])
@pytest.mark.parametrize("new", [26, 64])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_long_cache_is_cut_into_many_pieces_and_joined(kv_heads, new, dim, dtype):
    """Row blocks of 26 to 512 rows over 20,011 keys, shared out over all CTAs: up to 76 pieces a block."""
    ctx = 20011
    s = Step([ctx], [new], 8, kv_heads, dim, 32, dtype, "tree", seed=dim + new)
    out, lse = s.run(max_context=LONG)
    again, lse2 = s.run(max_context=LONG)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    on_tensor_cores(lambda: s.run(max_context=LONG), joined=True)
    # the reference of test_gpu_step.py, all rows of a head at once
    blocks = torch.as_tensor(s.table[0][:-(-(ctx + new) // 32)])
    k, v = (c[blocks].flatten(0, 1)[:ctx + new].double() for c in (s.k, s.v))
    seen = torch.ones((new, ctx + new), dtype=torch.bool)
    seen[:, ctx:] = torch.from_numpy(s.bits[:, :new])
    u = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    for h in range(8):
        g = h // (8 // kv_heads)
        a = (s.q[:, h].double() @ k[:, g].T * s.scale).masked_fill(~seen, -torch.inf)
        w = a.softmax(-1)
        close(out[:, h], w @ v[:, g], w @ v[:, g].abs(), u)
        want = a.logsumexp(-1)
        assert ((lse[:, h].double().cpu() - want).abs() <= 2.0 ** -13 * (1 + want.abs())).all()


@pytest.mark.parametrize("layout", ["heads_first", "blocks_last"])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_strides(layout, dim):
    """q as a part of a fused projection's rows, other orders of the cache's axes, a strided table."""
    s = Step([45, 100], [50, 20], 8, 2, dim, 32, torch.bfloat16, "tree", seed=dim)
    s.scale = 0.125
    fused = torch.zeros((s.T, 14, dim), dtype=torch.bfloat16, device="cuda")
    fused[:, 3:11] = s.q.cuda()
    if layout == "heads_first":
        k = s.k.cuda().transpose(1, 2).contiguous().transpose(1, 2)
        v = s.v.cuda().permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    else:
        k = s.k.cuda().permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)
        both = torch.zeros((*s.v.shape[:3], 2 * dim), dtype=torch.bfloat16, device="cuda")
        v = both[..., dim:]
        v.copy_(s.v)
    wide = torch.full((2, 40), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + s.table.shape[1]] = i32(s.table)
    lse = torch.empty((s.T, 8), device="cuda")
    call = lambda: awq.tree_attention(fused[:, 3:11], k, v, wide[:, 3:3 + s.table.shape[1]], i32(s.ctx), i32(s.cu), 0.125,  # noqa: E731
                                      50, LONG, tree_mask=s.mask.cuda(), lse=lse)
    s.check(call(), lse)
    on_tensor_cores(call)


@pytest.mark.parametrize("what", ["cu_decreases", "cu_past_end", "ctx_negative", "ctx_past_table", "page"])
def test_bad_lengths_and_pages_are_reported(what):
    s = Step([30, 40], [40, 30], 4, 2, 64, 16, torch.float16, "causal", garbage=0.0)
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
    call = lambda: awq.tree_attention(s.q.cuda(), s.k.cuda(), s.v.cuda(), i32(table), i32(ctx), i32(cu), 0.1, 40, LONG, out=out)  # noqa: E731
    call()
    on_tensor_cores(call)
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    if what != "page":
        assert (out == 5).all()
        return
    for b, page in ((1, 0), (0, 1)):                   # the pages read as zeros
        s.k[s.table[b, page]] = 0
        s.v[s.table[b, page]] = 0
    want, _, size = ref.attention(s.q, s.k, s.v, s.table, s.ctx, s.cu, 0.1, None)
    close(out, want, size)


@pytest.mark.parametrize("new", [[9, 1], [50, 70]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_odd_values_in_the_context_reach_every_row(new, bad):
    s = Step([37, 300], new, 8, 2, 64, 16, torch.float16, "tree")
    s.v[s.table[0][0], 3, 1, 7] = bad
    out, lse = s.run(max_context=LONG)
    on_tensor_cores(lambda: s.run(max_context=LONG))
    assert not out[:new[0], 4:, 7].isfinite().any()
    out[:new[0], 4:, 7] = 0
    assert out.isfinite().all() and lse.isfinite().all()


def test_own_streams_at_once():
    steps = [Step([3000 + 64 * i], [n], 8, 2, dim, 16, torch.float16, "tree", seed=i)
             for i, (n, dim) in enumerate([(9, 64), (33, 128), (70, 64), (40, 128)])]
    streams = [torch.cuda.Stream() for _ in steps]
    args = [(s.q.cuda(), s.k.cuda(), s.v.cuda(), i32(s.table), i32(s.ctx), i32(s.cu), s.mask.cuda()) for s in steps]
    torch.cuda.synchronize()
    outs = [[] for _ in steps]
    for _ in range(5):
        for s, st, a, o in zip(steps, streams, args, outs):
            with torch.cuda.stream(st):
                lse = torch.empty(s.q.shape[:2], device="cuda")
                o.append((awq.tree_attention(*a[:6], 0.125, max(s.new), LONG, tree_mask=a[6], lse=lse), lse))
    torch.cuda.synchronize()
    for s, o in zip(steps, outs):
        s.scale = 0.125
        s.check(*o[0])
        assert all(torch.equal(o[0][0], x) for x, _ in o[1:])


@pytest.mark.parametrize("mask", ["causal", "tree"])
def test_bounds_that_are_too_small(mask):
    """More rows than the bound: more blocks of 128. Longer caches than the bound: a CTA has all keys of a block."""
    s = Step([300, 10], [2, 70], 8, 2, 64, 16, torch.float16, mask)
    s.check(*s.run(max_new=17, max_context=LONG))
    on_tensor_cores(lambda: s.run(max_new=17, max_context=LONG), joined=True)
    rng = np.random.default_rng(1)
    ctx = [int(c) for c in rng.integers(0, 300, 80)]
    ctx[3] = 4100
    s = Step(ctx, [9] * 80, 16, 4, 64, 16, torch.float16, mask, seed=4)
    s.check(*s.run(max_context=50))
    on_tensor_cores(lambda: s.run(max_context=50), joined=False)


@pytest.mark.parametrize("new", [17, 80])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_chunk_of_a_long_prompt(new, dim):
    """No mask: each token sees the ones before it; its length passes several tiles and row blocks."""
    s = Step([0, 131, 5], [new * 5, new, 1], 4, 1, dim, 64, torch.bfloat16, "causal", seed=new)
    s.check(*s.run(max_context=LONG))
    on_tensor_cores(lambda: s.run(max_context=LONG))


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, its last block."""
    page, heads, dim = 1024, 8, 128
    blocks = 2 ** 32 // (page * heads * dim) + 3
    k = torch.zeros((blocks, page, heads, dim), dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    gen = torch.Generator().manual_seed(3)
    new_k, new_v = (torch.randn((200, heads, dim), generator=gen).half().cuda() for _ in range(2))
    awq.kv_append(new_k, new_v, k, v, (blocks - 1) * page + torch.arange(200, device="cuda"))
    q = torch.randn((40, 8, dim), generator=gen).half()
    call = lambda: awq.tree_attention(q.cuda(), k, v, i32([[blocks - 1]]), i32([160]), i32([0, 40]), 0.1, 40, LONG)  # noqa: E731
    want, _, size = ref.attention(q, new_k[None], new_v[None], np.array([[0]]), [160], [0, 40], 0.1)
    close(call(), want, size)
    on_tensor_cores(call)


def test_a_captured_call_follows_the_lengths():
    first = Step([900, 70], [33, 20], 8, 2, 128, 16, torch.float16, "tree", seed=1)
    later = Step([1333, 90], [20, 33], 8, 2, 128, 16, torch.float16, "tree", seed=2)
    stream = torch.cuda.Stream()
    assert awq.awq_reserve_tree_attention(128, stream.cuda_stream) == Status.OK
    with torch.cuda.stream(stream):
        q, mask = first.q.cuda(), first.mask.cuda()
        k = torch.zeros((later.k.shape[0], 16, 2, 128), dtype=torch.float16, device="cuda")
        v = torch.zeros_like(k)
        k[:first.k.shape[0]], v[:first.v.shape[0]] = first.k.cuda(), first.v.cuda()
        table = torch.full((2, later.table.shape[1]), -1, dtype=torch.int32, device="cuda")
        table[:, :first.table.shape[1]] = i32(first.table)
        ctx, cu = i32(first.ctx), i32(first.cu)
        out, lse = torch.empty_like(q), torch.empty((53, 8), device="cuda")
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream, capture_error_mode="global"):
        awq.tree_attention(q, k, v, table, ctx, cu, 0.125, 33, LONG, tree_mask=mask, out=out, lse=lse)
    first.scale = later.scale = 0.125
    graph.replay()
    torch.cuda.synchronize()
    first.check(out, lse)
    for dst, src in ((q, later.q), (k, later.k), (v, later.v), (mask, later.mask), (table, i32(later.table)),
                     (ctx, i32(later.ctx)), (cu, i32(later.cu))):
        dst.copy_(src)
    on_tensor_cores(graph.replay, joined=True)
    torch.cuda.synchronize()
    later.check(out, lse)


@pytest.mark.parametrize("requests,new,ctx,few", [(1, 64, 4000, False), (4, 16, 4000, False), (1, 32, 4000, True),
                                                  (1, 64, 2000, True), (16, 4, 2000, True), (16, 8, 400, False)])
def test_each_call_takes_the_faster_kernel(requests, new, ctx, few):
    """64 / 8 heads of 128: sizes at which the two kernels were timed against each other."""
    s = Step([ctx] * requests, [new] * requests, 64, 8, 128, 64, torch.float16, "tree")
    args = (s.q.cuda(), s.k.cuda(), s.v.cuda(), i32(s.table), i32(s.ctx), i32(s.cu), 0.1, new, ctx)
    mask = s.mask.cuda()
    names = kernels_of(lambda: awq.tree_attention(*args, tree_mask=mask))
    if names:
        assert any("attention_rows_kernel" in n for n in names) == few, names
