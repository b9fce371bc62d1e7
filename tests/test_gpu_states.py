"""GPU tests of reorder_states: outputs that lie between the states, rows without elements, views whose elements
are conjugated or negated only when they are read."""
import numpy as np
import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import Status

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status(gpu):
    """Every test starts and ends with a clean device status."""
    awq.awq_last_device_status(None)
    yield
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


def i32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


@pytest.mark.parametrize("from_,to", [
    (np.s_[:, 0], np.s_[:, 1]), (np.s_[:, 1], np.s_[:, 0]),          # beside each other in one allocation
    (np.s_[:, 0, 4:], np.s_[:, 0, :3]),                              # parts of one row
    (np.s_[::2, 0], np.s_[1::2, 1]),                                 # rows that alternate
    (np.s_[:9:4, 0], np.s_[1:8:2, 0]), (np.s_[8::3, 1], np.s_[::2, 0]),  # of different strides
    (np.s_[:3], np.s_[3:])])
def test_outputs_between_the_states(from_, to):
    buf = torch.arange(12 * 2 * 7, device="cuda", dtype=torch.int32).view(12, 2, 7)
    state, out = buf[from_], buf[to]
    parents = torch.randint(-1, state.shape[0], (out.shape[0],), device="cuda", dtype=torch.int32)
    want = torch.where((parents >= 0).view(-1, *[1] * (out.dim() - 1)), state[parents.clamp(min=0).long()], 0)
    rest = buf.clone()
    got, = awq.reorder_states([state], parents, outs=[out])
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)
    rest[to] = want
    assert torch.equal(buf, rest)


@pytest.mark.parametrize("from_,to", [
    (np.s_[:, 0, :4], np.s_[:, 0, 3:]), (np.s_[:, 0], np.s_[:, 0]), (np.s_[1:, 0], np.s_[:5, 0]),
    (np.s_[:9:4, 0], np.s_[::2, 0]),             # rows 0, 4, 8 and 0, 2, 4, ..
    (np.s_[1::3, 0], np.s_[::2, 0]),             # 1, 4, 7, 10 and 0, 2, 4, ..
    (np.s_[2:3], np.s_[:4])])
def test_outputs_that_overlap_the_states_are_refused(from_, to):
    buf = torch.zeros((12, 2, 7), device="cuda")
    with pytest.raises(ValueError):
        awq.reorder_states([torch.zeros((buf[from_].shape[0], 3), device="cuda"), buf[from_]],
                           torch.zeros(buf[to].shape[0], device="cuda", dtype=torch.int32),
                           outs=[torch.zeros((buf[to].shape[0], 3), device="cuda"), buf[to]])


def test_views_that_are_conjugated_or_negated_are_refused():
    z = torch.randn((4, 6), device="cuda", dtype=torch.complex64)
    parents = i32([3, 0])
    conjugate, negated = z.conj(), z.conj().imag
    assert conjugate.is_conj() and negated.is_neg()
    for view, plain in ((conjugate, conjugate.resolve_conj()), (negated, negated.resolve_neg())):
        with pytest.raises(ValueError):
            awq.reorder_states([view], parents)
        with pytest.raises(ValueError):
            awq.reorder_states([plain], parents, outs=[torch.empty_like(plain)[:2].conj() if plain.is_complex() else view[:2]])
        got, = awq.reorder_states([plain], parents)
        assert torch.equal(got, plain[[3, 0]])
    with pytest.raises(ValueError):
        awq.beam_select(negated, torch.zeros((1, 4), device="cuda"), 2)


@pytest.mark.parametrize("shape", [(0,), (3, 0), (0, 3), (2, 0, 5), (2, 5, 0)])
def test_rows_without_elements(shape):
    empty, full = torch.zeros((4, *shape), device="cuda"), torch.randn((4, 3), device="cuda")
    got, other = awq.reorder_states([empty, full], i32([3, 0, -1]))
    assert got.shape == (3, *shape) and torch.equal(other[:2], full[[3, 0]])
    outs = [torch.zeros((3, *shape), device="cuda"), torch.empty((3, 3), device="cuda")]
    awq.reorder_states([empty, full], i32([3, 0, -1]), outs=outs)
    assert torch.equal(outs[1], other)
