"""awq_reserve_tree_attention: what a stream holds afterwards, and which calls need nothing
of it. Tolerances as in test_gpu_step.py."""
import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
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


def on_the_gpu(s):
    s.scale = 0.1
    args = (s.q.cuda(), s.k.cuda(), s.v.cuda(), i32(s.table), i32(s.ctx), i32(s.cu), s.scale)
    kw = dict(tree_mask=s.mask.cuda(), out=torch.empty(s.q.shape, dtype=s.q.dtype, device="cuda"),
              lse=torch.empty(s.q.shape[:2], device="cuda"))
    torch.cuda.synchronize()
    return args, kw


def free_bytes():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]


@pytest.mark.parametrize("new", [1, 70])
def test_a_captured_call_outlives_a_larger_one(new):
    """A later call on the stream needs more scratch than was reserved: the graph's stays."""
    s = Step([20000], [new], 8, 2, 64, 32, torch.float16, "tree", seed=new)
    args, kw = on_the_gpu(s)
    big = Step([9000], [70], 8, 2, 128, 32, torch.float16, "tree", seed=7)
    big_args, big_kw = on_the_gpu(big)
    stream = torch.cuda.Stream()
    assert awq.awq_reserve_tree_attention(64, stream.cuda_stream) == Status.OK
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream, capture_error_mode="global"):
        awq.tree_attention(*args, new, LONG, **kw)
    before = free_bytes()
    with torch.cuda.stream(stream):
        awq.tree_attention(*big_args, 70, LONG, **big_kw)
    assert free_bytes() < before                       # it did need more
    big.check(big_kw["out"], big_kw["lse"])
    for _ in range(3):
        kw["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
            awq.tree_attention(*big_args, 70, LONG, **big_kw)
        stream.synchronize()
        s.check(kw["out"], kw["lse"])
        big.check(big_kw["out"], big_kw["lse"])


@pytest.mark.parametrize("reserved,dim", [(64, 8), (72, 128), (128, 64), (256, 64), (256, 128), (136, 256)])
@pytest.mark.parametrize("new", [1, 70])
def test_a_reservation_serves_smaller_head_dims(reserved, dim, new):
    """Neither kernel allocates: cut row blocks, pieces of every CTA."""
    s = Step([9000], [new], 8, 2, dim, 32, torch.float16, "tree", seed=dim)
    args, kw = on_the_gpu(s)
    stream = torch.cuda.Stream()
    assert awq.awq_reserve_tree_attention(reserved, stream.cuda_stream) == Status.OK
    before = free_bytes()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        awq.tree_attention(*args, new, LONG, **kw)
    assert free_bytes() == before
    s.check(kw["out"], kw["lse"])
    kw["out"].fill_(float("nan"))
    with torch.cuda.graph(graph, stream=stream, capture_error_mode="global"):
        awq.tree_attention(*args, new, LONG, **kw)
    graph.replay()
    torch.cuda.synchronize()
    s.check(kw["out"], kw["lse"])


@pytest.mark.parametrize("ctx,new,heads,kv_heads", [(100, 1, 4, 4), (900, 1, 32, 4), (900, 20, 64, 8), (0, 1, 1, 1),
                                                    (0, 70, 8, 1)])
def test_calls_that_cut_no_row_block_need_no_scratch(ctx, new, heads, kv_heads):
    """Short caches, on a stream that holds nothing: nothing is allocated, so they can be captured."""
    s = Step([ctx] * 2, [new] * 2, heads, kv_heads, 128, 32, torch.float16, "tree", seed=heads)
    args, kw = on_the_gpu(s)
    with torch.cuda.stream(torch.cuda.Stream()):       # the kernels' code is on the GPU after this
        awq.tree_attention(*args, new, ctx, **kw)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    before = free_bytes()
    with torch.cuda.stream(stream):
        awq.tree_attention(*args, new, ctx, **kw)
    assert free_bytes() == before
    with torch.cuda.graph(graph, stream=stream, capture_error_mode="global"):
        awq.tree_attention(*args, new, ctx, **kw)
    kw["out"].fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    s.check(kw["out"], kw["lse"])
