"""What beam_select leaves where a wait for its logits runs out (the fault-test build, include/awq_gb300_fault_test.h):
the rows whose logits did not come have no candidates. Tokens and parents go on into the next step before
anyone reads the device status, so they are in range whatever the workspace held before."""
import ctypes

import pytest
import torch

from bit_weight_quantized_awq_gb300 import BeamSelect, Status
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
    lib.awq_last_device_status.argtypes = [P]
    lib.awq_test_inject_fault.argtypes = [ctypes.c_int]
    lib.awq_test_inject_fault.restype = None
    yield lib
    lib.awq_test_inject_fault(0)


# a word that a list would take for the logit -0.25 of token 1027080191, and the sums for 16 e^-100: the best by far
STALE = 0x41800000C2C80000


class Call:
    def __init__(self, flib, B, W, V, keep, dtype):
        self.flib, self.B, self.W, self.V = flib, B, W, V
        gen = torch.Generator(device="cuda").manual_seed(V)
        self.logits = torch.randn((B * W, V), device="cuda", generator=gen).to(dtype)
        self.before = -torch.rand((B, W), device="cuda", generator=gen)
        self.ends = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
        code = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}[dtype]
        size = flib.awq_beam_select_workspace(B, W, V, keep, 2, code)
        self.space = torch.full((size // 8,), STALE, dtype=torch.int64, device="cuda")
        self.out = [torch.zeros((B, keep), device="cuda", dtype=torch.int32 if i % 3 else torch.float32) for i in range(6)]
        p = [t.data_ptr() for t in self.out]
        self.args = BeamSelect(logits=self.logits.data_ptr(), logits_row_stride=V, requests=B, beams=W, vocab=V,
                               scores=self.before.data_ptr(), num_beams=keep, end_tokens=self.ends.data_ptr(), num_ends=2,
                               out_scores=p[0], out_parents=p[1], out_tokens=p[2], ended_scores=p[3], ended_parents=p[4],
                               ended_tokens=p[5], workspace=self.space.data_ptr(), workspace_bytes=size, dtype=code)

    def __call__(self):
        assert self.flib.awq_beam_select(ctypes.byref(self.args), torch.cuda.current_stream().cuda_stream) == Status.OK
        torch.cuda.synchronize()

    def status(self):
        return self.flib.awq_last_device_status(torch.cuda.current_stream().cuda_stream)

    def in_range(self):
        row = torch.arange(self.B, device="cuda")[:, None]
        for s, p, t in (self.out[:3], self.out[3:]):
            none = p == -1
            assert (none == (t == -1)).all() and (none | ((p // self.W == row) & (t >= 0) & (t < self.V))).all()
            assert (s[none] == -torch.inf).all() and not torch.isnan(s).any()


# a part of a row, some rows, one long row of which CTA 0 has a part, several rows a CTA
SIZES = [(2, 3, 50000, 4, torch.float16), (2, 3, 700, 4, torch.float32), (1, 3, 2000003, 4, torch.bfloat16),
         (300, 3, 700, 8, torch.float16), (77, 8, 70003, 8, torch.bfloat16)]


@pytest.mark.parametrize("B,W,V,keep,dtype", SIZES)
def test_rows_whose_logits_do_not_come_have_no_candidates(flib, B, W, V, keep, dtype):
    call = Call(flib, B, W, V, keep, dtype)
    assert call.status() == Status.OK
    flib.awq_test_inject_fault(1)
    try:
        call()
    finally:
        flib.awq_test_inject_fault(0)
    assert call.status() == Status.ERR_TIMEOUT
    call.in_range()
    assert not (call.out[1] == 0).any()                # row 0 is CTA 0's
    failed = [t.clone() for t in call.out]
    call()
    assert call.status() == Status.OK
    call.in_range()
    # requests that CTA 0 has no part of are as they should be
    for a, b in zip(failed, call.out):
        assert torch.equal(a[B // 2 + 1:], b[B // 2 + 1:])


@pytest.mark.parametrize("B,W,V,keep,dtype", SIZES)
def test_copies_land_before_a_row_that_was_given_up_ends(flib, B, W, V, keep, dtype):
    """The working warps leave while copies are under way; the producer waits for those. Shares that fit the ring
    and longer ones."""
    call = Call(flib, B, W, V, keep, dtype)
    call()
    right = [t.clone() for t in call.out]
    for _ in range(5):
        call.space.fill_(STALE)
        flib.awq_test_inject_fault(2)
        try:
            call()
        finally:
            flib.awq_test_inject_fault(0)
        assert call.status() == Status.ERR_TIMEOUT
        call.in_range()
        assert not (call.out[1] == 0).any()
        call()
        assert call.status() == Status.OK and all(torch.equal(a, b) for a, b in zip(call.out, right))
