"""The tree-attention kernels' bounded waits, made to run out on purpose without a
GPU fault (the fault-test build, include/awq_gb300_fault_test.h): CTA 0's producers
issue no copy, so its waits run out after about 2 ms. The call returns, the device
status says AWQ_ERR_TIMEOUT, and the next calls on the same stream are right."""
import ctypes

import pytest
import torch

import step_reference as ref
from bit_weight_quantized_awq_gb300 import Status, TreeAttention, Cache
from bit_weight_quantized_awq_gb300.build import FAULT_LIB, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def flib(gpu):
    build(quiet=True)
    lib = ctypes.CDLL(FAULT_LIB)
    lib.awq_tree_attention.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.awq_last_device_status.argtypes = [ctypes.c_void_p]
    lib.awq_test_inject_fault.argtypes = [ctypes.c_int]
    lib.awq_test_inject_fault.restype = None
    yield lib
    lib.awq_test_inject_fault(0)


@pytest.mark.parametrize("ctx,new,dim", [(500, 1, 128), (900, 1, 256), (300, 2, 64)])
def test_wait_of_a_cluster_runs_out_then_next_calls_are_right(flib, ctx, new, dim):
    """Short row blocks, which the CTAs of a cluster share: all of them leave."""
    _runs_out(flib, ctx, new, dim)


@pytest.mark.parametrize("new,dim", [(12, 64), (40, 128), (80, 128)])
def test_wait_of_the_tensor_core_kernel_runs_out_then_next_calls_are_right(flib, new, dim):
    """Bounds that allow a long cache, for which that kernel is taken."""
    _runs_out(flib, 2001, new, dim, max_context=2 ** 20)


@pytest.mark.parametrize("new,dim", [(1, 128), (1, 256), (12, 64), (40, 128), (80, 128)])
def test_wait_runs_out_then_next_calls_are_right(flib, new, dim):
    _runs_out(flib, 2001, new, dim)


def _runs_out(flib, ctx, new, dim, max_context=None):
    gen = torch.Generator().manual_seed(new + dim)
    page = 32
    blocks = -(-(ctx + new) // page)
    q = torch.randn((new, 8, dim), generator=gen).half()
    k, v = (torch.randn((blocks, page, 2, dim), generator=gen).half() for _ in range(2))
    table = torch.randperm(blocks, generator=gen).to(torch.int32)[None]
    dev = [t.cuda() for t in (q, k, v, table, torch.tensor([ctx], dtype=torch.int32),
                              torch.tensor([0, new], dtype=torch.int32))]
    out = torch.empty_like(dev[0])
    cache = lambda t: Cache(t.data_ptr(), page * 2 * dim, 2 * dim, dim)  # noqa: E731
    args = TreeAttention(dev[0].data_ptr(), 8 * dim, dim, out.data_ptr(), None, cache(dev[1]), cache(dev[2]),
                         dev[3].data_ptr(), blocks, blocks, dev[4].data_ptr(), dev[5].data_ptr(), None, 0, 1, new, 8,
                         2, dim, blocks, page, new, max_context or ctx, 0.1, 0)
    stream = torch.cuda.current_stream().cuda_stream
    call = lambda: flib.awq_tree_attention(ctypes.byref(args), stream)  # noqa: E731
    assert flib.awq_last_device_status(stream) == Status.OK
    flib.awq_test_inject_fault(1)
    try:
        assert call() == Status.OK
    finally:
        flib.awq_test_inject_fault(0)
    assert flib.awq_last_device_status(stream) == Status.ERR_TIMEOUT
    want, _, size = ref.attention(q, k, v, table.numpy(), [ctx], [0, new], 0.1)
    for _ in range(2):
        out.fill_(float("nan"))
        assert call() == Status.OK
        torch.cuda.synchronize()
        err = (out.double().cpu() - want).abs()
        assert (err <= 2.0 ** -11 * want.abs() + (2.0 ** -11 + 2.0 ** -13) * size + 2.0 ** -24).all()
    assert flib.awq_last_device_status(stream) == Status.OK
