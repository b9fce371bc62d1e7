"""The bounded waits of beam_select's rows and of the bulk copies of pages, made to run out on
purpose without a GPU fault (the fault-test build, include/awq_gb300_fault_test.h): CTA 0 issues no
copy, so its waits run out after about 2 ms. The calls return, the device status says
AWQ_ERR_TIMEOUT, and the next calls on the same stream are right."""
import ctypes

import pytest
import torch

import beam_reference as ref
from bit_weight_quantized_awq_gb300 import BeamSelect, Cache, Status
from bit_weight_quantized_awq_gb300.build import FAULT_LIB, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def flib(gpu):
    build(quiet=True)
    lib = ctypes.CDLL(FAULT_LIB)
    P, I = ctypes.c_void_p, ctypes.c_int64
    lib.awq_beam_select.argtypes = [P, P]
    lib.awq_beam_select_workspace.argtypes = [I, I, I, I, I, ctypes.c_int]
    lib.awq_beam_select_workspace.restype = I
    lib.awq_copy_pages.argtypes = [P, I, P, I, I, I, I, P, P, P, I, P, P]
    lib.awq_last_device_status.argtypes = [P]
    lib.awq_test_inject_fault.argtypes = [ctypes.c_int]
    lib.awq_test_inject_fault.restype = None
    yield lib
    lib.awq_test_inject_fault(0)


def runs_out(flib, call, right):
    stream = torch.cuda.current_stream().cuda_stream
    assert flib.awq_last_device_status(stream) == Status.OK
    flib.awq_test_inject_fault(1)
    try:
        assert call(stream) == Status.OK
    finally:
        flib.awq_test_inject_fault(0)
    assert flib.awq_last_device_status(stream) == Status.ERR_TIMEOUT
    for _ in range(2):
        assert call(stream) == Status.OK
        torch.cuda.synchronize()
        right()
    assert flib.awq_last_device_status(stream) == Status.OK


@pytest.mark.parametrize("vocab,dtype", [(50000, torch.float16), (700, torch.float32), (2000003, torch.bfloat16)])
def test_wait_of_the_logits_runs_out_then_next_calls_are_right(flib, vocab, dtype):
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    logits = torch.randn((6, vocab), device="cuda", generator=gen).to(dtype)
    before = torch.tensor([[-1.0, -2.5, -4.0], [-3.0, -1.25, -9.0]], device="cuda")
    code = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}[dtype]
    size = flib.awq_beam_select_workspace(2, 3, vocab, 4, 0, code)
    space = torch.zeros(size, dtype=torch.uint8, device="cuda")
    scores, parents, tokens = torch.zeros((2, 4), device="cuda"), *(torch.zeros((2, 4), dtype=torch.int32, device="cuda") for _ in range(2))
    args = BeamSelect(logits=logits.data_ptr(), logits_row_stride=vocab, requests=2, beams=3, vocab=vocab, scores=before.data_ptr(),
                      num_beams=4, out_scores=scores.data_ptr(), out_parents=parents.data_ptr(), out_tokens=tokens.data_ptr(),
                      workspace=space.data_ptr(), workspace_bytes=size, dtype=code)
    live, _ = ref.beams(logits.double().cpu().numpy(), before.cpu().numpy(), 4)

    def right():
        for b in range(2):
            assert list(zip(parents[b].tolist(), tokens[b].tolist())) == [w[1:] for w in live[b]]
    runs_out(flib, lambda stream: flib.awq_beam_select(ctypes.byref(args), stream), right)


def test_wait_of_a_bulk_copy_runs_out_then_next_calls_are_right(flib):
    cache = torch.randn((300, 64, 8, 128), device="cuda").half()
    perm = torch.randperm(300, device="cuda").int()
    src, dst = perm[:150].contiguous(), perm[150:].contiguous()
    layout = Cache(cache.data_ptr(), 64 * 8 * 128, 8 * 128, 128)
    pointers = (ctypes.c_void_p * 1)(cache.data_ptr())
    call = lambda stream: flib.awq_copy_pages(pointers, 1, ctypes.byref(layout), 300, 64, 8, 128, src.data_ptr(),  # noqa: E731
                                              dst.data_ptr(), None, 150, None, stream)

    def right():
        assert torch.equal(cache[dst.long()], cache[src.long()])
    runs_out(flib, call, right)
