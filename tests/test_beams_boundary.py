"""Host-only checks of the entry points of rotary positions, beam search and a cache's pages: every
refusal comes before any CUDA call, so these run without a GPU."""
import ctypes

import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import BeamSelect, Cache, Rotary, State, Status
from bit_weight_quantized_awq_gb300.build import build

A = 0x10000      # 16-byte aligned fake device address: never dereferenced here
INVALID, MISALIGNED, OK = Status.ERR_INVALID_ARG, Status.ERR_MISALIGNED, Status.OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    build(quiet=True)
    return awq.load_library()


def cache(**k):
    return Cache(**dict(dict(data=A, block_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64), **k))


def rotary(**k):
    d = dict(q=A, k=A, v=A, q_token_stride=256, q_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128,
             v_head_stride=64, q_out=A + 0x1000, k_out=A + 0x2000, q_out_token_stride=256, q_out_head_stride=64,
             k_out_token_stride=128, k_out_head_stride=64, positions=A, inv_freq=A, axes=None, tokens=3, q_heads=4,
             kv_heads=2, head_dim=64, rotary_dim=64, num_axes=1, pairs=0, dtype=0)
    d.update(k)
    return awq.awq_rotary(Rotary(**d), None)


APPEND = dict(slot_map=A, k_cache=cache(), v_cache=cache(), num_blocks=4, block_size=16)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dtype=-1), dict(tokens=-1), dict(tokens=2 ** 31), dict(q_heads=0), dict(kv_heads=-1), dict(head_dim=12),
    dict(head_dim=0), dict(head_dim=1032), dict(rotary_dim=0), dict(rotary_dim=63), dict(rotary_dim=66), dict(num_axes=0),
    dict(q_heads=2 ** 18), dict(q_token_stride=4), dict(k_head_stride=-8), dict(q_out_token_stride=1), dict(v_token_stride=3),
    dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(positions=None), dict(inv_freq=None),
    dict(q_out=A, q_out_token_stride=512), dict(k_out=A, k_out_head_stride=128), dict(q_token_stride=2 ** 38),
    dict(APPEND, v=None), dict(APPEND, kv_heads=0), dict(APPEND, block_size=24), dict(APPEND, num_blocks=-1),
    dict(APPEND, k_cache=cache(data=None)), dict(APPEND, v_cache=cache(token_stride=4)), dict(APPEND, k_cache=cache(block_stride=0))])
def test_rotary_invalid(kw):
    assert rotary(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(q=A + 8), dict(k=A + 2), dict(q_out=A + 4), dict(k_out=A + 8), dict(positions=A + 2),
                                dict(inv_freq=A + 1), dict(axes=A + 2), dict(APPEND, slot_map=A + 4), dict(APPEND, v=A + 8),
                                dict(APPEND, v_cache=cache(data=A + 8))])
def test_rotary_misaligned(kw):
    assert rotary(**kw) == MISALIGNED


def test_rotary_empty():
    assert rotary(tokens=0, q=None, k=None, positions=None) == OK
    assert awq.awq_rotary(None, None) == INVALID


def beam(**k):
    d = dict(logits=A, logits_row_stride=100, requests=2, beams=4, vocab=100, scores=A, num_beams=4, end_tokens=A, num_ends=1,
             out_scores=A, out_parents=A, out_tokens=A, ended_scores=A, ended_parents=A, ended_tokens=A, workspace=A,
             workspace_bytes=1 << 20, dtype=0)
    d.update(k)
    return awq.awq_beam_select(BeamSelect(**d), None)


@pytest.mark.parametrize("kw", [
    dict(requests=-1), dict(requests=16385), dict(beams=0), dict(beams=33), dict(num_beams=0), dict(num_beams=33), dict(num_ends=-1),
    dict(num_ends=9), dict(vocab=0), dict(vocab=2 ** 27 + 1), dict(dtype=3), dict(dtype=-1), dict(end_tokens=None),
    dict(logits_row_stride=99), dict(logits=None), dict(scores=None), dict(out_scores=None), dict(out_parents=None),
    dict(out_tokens=None), dict(ended_scores=None), dict(ended_parents=None), dict(ended_tokens=None), dict(workspace=None),
    dict(workspace_bytes=8)])
def test_beam_select_invalid(kw):
    assert beam(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(logits=A + 1), dict(logits=A + 2, dtype=2), dict(workspace=A + 16), dict(scores=A + 2),
                                dict(end_tokens=A + 1), dict(out_scores=A + 2), dict(ended_tokens=A + 2)])
def test_beam_select_misaligned(kw):
    assert beam(**kw) == MISALIGNED


def test_beam_select_without_end_tokens():
    none = dict(end_tokens=None, num_ends=0)
    assert beam(**none, ended_parents=None) == INVALID and beam(**none, ended_scores=None, workspace=None) == INVALID


def test_beam_select_empty_and_workspace():
    assert beam(requests=0, logits=None, scores=None, workspace=None) == OK
    assert awq.awq_beam_select(None, None) == INVALID
    size = awq.awq_beam_select_workspace
    assert size(0, 4, 100, 4, 0, 0) == 0 and size(1, 4, 32000, 4, 1, 0) > 0
    for bad in ((-1, 4, 100, 4, 0, 0), (1, 33, 100, 4, 0, 0), (1, 4, 0, 4, 0, 0), (1, 4, 100, 0, 0, 0), (1, 4, 100, 4, 9, 0),
                (1, 4, 100, 4, 0, 3)):
        assert size(*bad) == -1
    need = size(2, 4, 100, 4, 1, 0)
    assert beam(workspace_bytes=need - 1) == INVALID


def states(*items):
    return (State * len(items))(*(State(**dict(dict(src=A, dst=A + 0x1000, src_row_stride=64, dst_row_stride=64, row_bytes=64), **i))
                                  for i in items))


def test_reorder_states():
    call = awq.awq_reorder_states
    assert call(None, 1, A, 2, 2, None) == INVALID and call(states({}), -1, A, 2, 2, None) == INVALID
    assert call(states({}), 4097, A, 2, 2, None) == INVALID and call(states({}), 1, None, 2, 2, None) == INVALID
    assert call(states({}), 1, A, -1, 2, None) == INVALID and call(states({}), 1, A, 2, 2 ** 31, None) == INVALID
    for bad in (dict(row_bytes=-1), dict(row_bytes=2 ** 31), dict(src_row_stride=63), dict(dst_row_stride=0), dict(src=None),
                dict(dst=None), dict(src_row_stride=2 ** 40)):
        assert call(states({}, bad), 2, A, 2, 2, None) == INVALID
    assert call(states({}), 1, A + 2, 2, 2, None) == MISALIGNED
    assert call(None, 0, None, 2, 2, None) == OK and call(states({}), 1, None, 0, 2, None) == OK


def fork(**k):
    d = dict(table=A, rows_in=2, width=8, stride=8, lens=A, parents=A, rows_out=3, free=A, num_free=4, start=None, page=16,
             new=A + 0x1000, new_stride=8, new_lens=A, src=A, dst=A, tokens=A, count=A)
    d.update(k)
    return awq.awq_fork_pages(*d.values(), None)


@pytest.mark.parametrize("kw", [
    dict(rows_in=-1), dict(rows_in=16385), dict(rows_out=-1), dict(rows_out=16385), dict(page=8), dict(page=48), dict(width=0),
    dict(width=2 ** 30 + 1, stride=2 ** 31, new_stride=2 ** 31), dict(stride=7), dict(new_stride=7), dict(num_free=-1),
    dict(num_free=2 ** 31), dict(table=None), dict(lens=None), dict(parents=None), dict(free=None), dict(new=None),
    dict(new_lens=None), dict(src=None), dict(dst=None), dict(tokens=None), dict(count=None), dict(new=A)])
def test_fork_invalid(kw):
    assert fork(**kw) == INVALID


@pytest.mark.parametrize("name", ["table", "lens", "parents", "free", "start", "new", "new_lens", "src", "dst", "tokens", "count"])
def test_fork_misaligned(name):
    assert fork(**{name: A + 2}) == MISALIGNED


def copy(**k):
    d = dict(caches=(ctypes.c_void_p * 2)(A, A), n=2, layout=cache(), blocks=4, page=16, heads=2, dim=64, src=A, dst=A, tokens=None,
             pairs=3, count=None)
    d.update(k)
    return awq.awq_copy_pages(*d.values(), None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=65537), dict(pairs=-1), dict(pairs=2 ** 31), dict(blocks=0), dict(blocks=2 ** 31), dict(page=17), dict(heads=0),
    dict(dim=12), dict(dim=0), dict(heads=2 ** 19, dim=1024), dict(layout=None), dict(layout=cache(token_stride=4)),
    dict(layout=cache(head_stride=0)), dict(caches=None), dict(caches=(ctypes.c_void_p * 2)(A, None)), dict(src=None), dict(dst=None)])
def test_copy_invalid(kw):
    assert copy(**kw) == INVALID


def test_copy_misaligned_and_empty():
    assert copy(caches=(ctypes.c_void_p * 2)(A, A + 8)) == MISALIGNED
    for name in ("src", "dst", "tokens", "count"):
        assert copy(**{name: A + 2}) == MISALIGNED
    assert copy(n=0, caches=None) == OK and copy(pairs=0, src=None, dst=None) == OK


def free(**k):
    d = dict(table=A, rows=2, width=8, stride=8, lens=A, page=16, blocks=100, held=None, num_held=0, free=A, counts=A, workspace=A)
    d.update(k)
    return awq.awq_free_pages(*d.values(), None)


def compact(**k):
    d = dict(table=A, rows=2, width=8, stride=8, lens=A, page=16, blocks=100, held=None, num_held=0, new=A + 0x1000, new_stride=8,
             map=A, src=A, dst=A, count=A, workspace=A)
    d.update(k)
    return awq.awq_compact_pages(*d.values(), None)


@pytest.mark.parametrize("call", [free, compact])
@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=2 ** 20 + 1), dict(width=0), dict(width=2 ** 30 + 1, stride=2 ** 31, new_stride=2 ** 31), dict(stride=7),
    dict(page=8), dict(page=100), dict(blocks=0),
    dict(blocks=2 ** 28 + 1), dict(num_held=-1), dict(num_held=1), dict(table=None), dict(lens=None), dict(workspace=None)])
def test_pages_invalid(call, kw):
    if call is free:
        kw = {k: v for k, v in kw.items() if k != "new_stride"}
    assert call(**kw) == INVALID


def test_pages_outputs():
    for kw in (dict(free=None), dict(counts=None)):
        assert free(**kw) == INVALID
    for kw in (dict(new=None), dict(new=A), dict(map=None), dict(src=None), dict(dst=None), dict(count=None), dict(new_stride=7)):
        assert compact(**kw) == INVALID
    for name in ("table", "lens", "free", "counts"):
        assert free(**{name: A + 2}) == MISALIGNED
    for name in ("table", "lens", "new", "map", "src", "dst", "count"):
        assert compact(**{name: A + 2}) == MISALIGNED
    for call in (free, compact):
        assert call(workspace=A + 128) == MISALIGNED and call(held=A + 2, num_held=1) == MISALIGNED
    size = awq.awq_pages_workspace
    assert size(0) == -1 and size(2 ** 28 + 1) == -1 and size(1) > 0 and size(2 ** 28) >= 2 ** 26


def test_wrappers_refuse_cpu_tensors():
    f, i = torch.zeros((2, 4, 64), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    c = torch.zeros((3, 16, 4, 64), dtype=torch.float16)
    for call in (lambda: awq.rotary(f, f, i, torch.zeros(32)), lambda: awq.rotary_append(f, f, f, i, torch.zeros(32), c, c, i.long()),
                 lambda: awq.beam_select(torch.zeros((2, 10)), torch.zeros((1, 2)), 2), lambda: awq.reorder_states([f], i),
                 lambda: awq.fork_pages(i[None], i[:1], i, i, 16), lambda: awq.copy_pages([c], i, i),
                 lambda: awq.free_pages(i[None], i[:1], 16, 9), lambda: awq.compact_pages(i[None], i[:1], 16, 9)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2,
                    reason="where torch sees a GPU, a fake tensor of cuda:1 needs a second one")
def test_wrappers_refuse_tensors_of_another_than_the_current_device():
    """Fake tensors, which have a device but no memory: refused before anything asks for it."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        make = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="cuda:1")  # noqa: E731
        i, table, slots, x = make(2), make(2, 4), make(2, dtype=torch.int64), make(2, 10, dtype=torch.float32)
        q, c, f = make(2, 4, 64, dtype=torch.float16), make(3, 16, 4, 64, dtype=torch.float16), make(32, dtype=torch.float32)
    for call in (lambda: awq.rotary(q, q, i, f), lambda: awq.rotary_append(q, q, q, i, f, c, c, slots),
                 lambda: awq.beam_select(x, f.view(1, 32)[:, :2], 2), lambda: awq.reorder_states([x], i),
                 lambda: awq.fork_pages(table, i, i, i, 16), lambda: awq.copy_pages([c], i, i),
                 lambda: awq.free_pages(table, i, 16, 9), lambda: awq.compact_pages(table, i, 16, 9)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
