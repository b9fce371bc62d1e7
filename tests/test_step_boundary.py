"""Host-only checks of the decoding step's entry points: every refusal comes
before any CUDA call, so these run without a GPU."""
import os
import subprocess
import sys

import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import Cache, Logits, Status, TreeAttention
from bit_weight_quantized_awq_gb300.build import build

A = 0x10000      # 16-byte aligned fake device address: never dereferenced here
INVALID, MISALIGNED, OK = Status.ERR_INVALID_ARG, Status.ERR_MISALIGNED, Status.OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    build(quiet=True)
    return awq.load_library()


def plan(**k):
    d = dict(ctx=A, new=A, B=2, table=A, width=8, stride=8, free=A, num_free=4, page=16, parents=None, tokens=9,
             cu=A, slots=A, pos=A, req=A, mask=None, words=0, counts=A)
    d.update(k)
    return awq.awq_paged_plan(*d.values(), None)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(B=16385), dict(page=8), dict(page=24), dict(page=2048), dict(page=0), dict(tokens=-1),
    dict(tokens=2 ** 30 + 1), dict(width=0), dict(stride=7), dict(num_free=-1), dict(words=-1), dict(words=1025),
    dict(words=1), dict(ctx=None), dict(new=None), dict(table=None), dict(free=None), dict(cu=None),
    dict(slots=None), dict(pos=None), dict(req=None), dict(counts=None)])
def test_plan_invalid(kw):
    assert plan(**kw) == INVALID


@pytest.mark.parametrize("name", ["ctx", "new", "table", "free", "parents", "cu", "pos", "req", "counts"])
def test_plan_misaligned(name):
    assert plan(**{name: A + 2}) == MISALIGNED
    assert plan(slots=A + 4) == MISALIGNED


def cache(**k):
    d = dict(data=A, block=16 * 2 * 64, token=2 * 64, head=64)
    d.update(k)
    return Cache(*d.values())


def append(**k):
    d = dict(k=A, kt=128, kh=64, v=A, vt=128, vh=64, kc=cache(), vc=cache(), slots=A, tokens=3, blocks=4, page=16,
             heads=2, dim=64)
    d.update(k)
    return awq.awq_kv_append(*d.values(), None)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(blocks=-1), dict(page=17), dict(heads=0), dict(dim=0), dict(dim=12), dict(kt=12),
    dict(vh=4), dict(kc=cache(block=4)), dict(vc=cache(head=0)), dict(k=None), dict(v=None), dict(slots=None),
    dict(kc=cache(data=None)), dict(kc=None), dict(kt=-8)])
def test_append_invalid(kw):
    assert append(**kw) == INVALID


def test_append_misaligned_and_empty():
    assert append(k=A + 8) == MISALIGNED
    assert append(vc=cache(data=A + 8)) == MISALIGNED
    assert append(slots=A + 4) == MISALIGNED
    assert append(tokens=0, k=None, v=None, slots=None) == OK


def attention(**k):
    d = dict(q=A, q_token_stride=256, q_head_stride=64, out=A, lse=None, k_cache=cache(), v_cache=cache(),
             block_table=A, table_width=8, table_stride=8, context_lens=A, cu_new=A, tree_mask=None, mask_words=0,
             B=1, tokens=2, q_heads=4, kv_heads=2, head_dim=64, num_blocks=4, block_size=16, max_new=2,
             max_context=10, scale=1.0, dtype=0)
    d.update(k)
    return awq.awq_tree_attention(TreeAttention(**d), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dtype=-1), dict(B=-1), dict(B=16385), dict(tokens=-1), dict(q_heads=0), dict(kv_heads=0),
    dict(q_heads=5), dict(head_dim=12), dict(head_dim=264), dict(head_dim=0), dict(num_blocks=0),
    dict(block_size=20), dict(block_size=8), dict(max_new=-1), dict(max_context=-1), dict(table_width=0),
    dict(table_stride=7), dict(tree_mask=A), dict(q_token_stride=4), dict(q_head_stride=1), dict(q=None),
    dict(out=None), dict(block_table=None), dict(context_lens=None), dict(cu_new=None),
    dict(k_cache=cache(data=None)), dict(k_cache=cache(token=12)), dict(v_cache=cache(head=2 ** 40)),
    dict(tokens=2 ** 30), dict(table_width=2 ** 28, table_stride=2 ** 28)])
def test_attention_invalid(kw):
    assert attention(**kw) == INVALID


def test_attention_rows_limit():
    # rows (tokens * group) are rounded up to whole blocks in 32 bits
    wide = dict(q_heads=2, kv_heads=1, q_token_stride=128, B=0)
    assert attention(tokens=2 ** 30 - 1, **wide) == INVALID
    assert attention(tokens=2 ** 30 - 512, **wide) == INVALID
    assert attention(tokens=2 ** 30 - 513, **wide) == OK


def test_attention_misaligned_and_empty():
    assert attention(q=A + 8) == MISALIGNED
    assert attention(out=A + 2) == MISALIGNED
    assert attention(v_cache=cache(data=A + 8)) == MISALIGNED
    assert attention(cu_new=A + 1) == MISALIGNED
    assert attention(tree_mask=A + 2, mask_words=1) == MISALIGNED
    assert attention(tokens=0, q=None, out=None) == OK
    assert attention(B=0, context_lens=None) == OK
    assert awq.awq_tree_attention(None, None) == INVALID


@pytest.mark.parametrize("head_dim", [0, -64, 65, 264, 2 ** 40])
def test_reserve_invalid(head_dim):
    assert awq.awq_reserve_tree_attention(head_dim, None) == INVALID


def logits(**k):
    d = dict(logits=A, out=A, logits_row_stride=100, out_row_stride=100, rows=2, vocab=100, B=2, dtype=0)
    d.update(k)
    return awq.awq_process_logits(Logits(**d), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(rows=-1), dict(vocab=0), dict(vocab=2 ** 27 + 1), dict(B=-1), dict(history=A),
    dict(draft_tokens=A), dict(bias_tokens=A), dict(bias_values=A), dict(bias_tokens=A, bias_values=A),
    dict(logits_row_stride=99), dict(out_row_stride=50), dict(out_row_stride=101), dict(logits=None),
    dict(out=None), dict(history_size=-1), dict(grammar_count=-1), dict(draft_tokens=A, cu_new=A, tree_mask=A)])
def test_logits_invalid(kw):
    assert logits(**kw) == INVALID


def test_logits_history_limit():
    # a counter keeps a token's occurrences in 30 bits
    assert logits(history=A, history_offsets=A, history_size=2 ** 29) == INVALID
    assert logits(history=A, history_offsets=A, history_size=2 ** 29 - 1, rows=0) == OK


def test_logits_bias_limit():
    # a thread's first pairs are numbered from the list's beginning in 32 bits: 2^31 less a few would wrap
    lists = dict(bias_tokens=A, bias_values=A, bias_offsets=A)
    for size in (2 ** 31 - 1, 2 ** 30 + 1):
        assert logits(bias_size=size, **lists) == INVALID
    assert logits(bias_size=2 ** 30, rows=0, **lists) == OK


def test_logits_misaligned_and_empty():
    assert logits(logits=A + 1, out=A + 4) == MISALIGNED
    assert logits(logits=A + 2, out=A + 4, dtype=2) == MISALIGNED
    assert logits(row_request=A + 2) == MISALIGNED
    assert logits(rows=0, logits=None, out=None) == OK
    assert awq.awq_process_logits(None, None) == INVALID


def test_wrappers_refuse_cpu_tensors():
    f, i = torch.zeros((2, 4, 64), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    c = torch.zeros((3, 16, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        awq.paged_plan(i, i, i[None], i, 16, 2)
    with pytest.raises(ValueError):
        awq.kv_append(f, f, c, c, i.long())
    with pytest.raises(ValueError):
        awq.tree_attention(f, c, c, i[None], i[:1], i, 1.0, 2, 0)
    with pytest.raises(ValueError):
        awq.process_logits(torch.zeros((2, 10)))


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2,
                    reason="where torch sees a GPU, a fake tensor of cuda:1 needs a second one")
def test_wrappers_refuse_tensors_of_another_than_the_current_device():
    """Fake tensors, which have a device but no memory: refused before anything asks for it."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        make = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="cuda:1")  # noqa: E731
        i, table, slots = make(2), make(2, 4), make(2, dtype=torch.int64)
        q, cache = make(2, 4, 64, dtype=torch.float16), make(3, 16, 4, 64, dtype=torch.float16)
        x = make(2, 10, dtype=torch.float32)
    for call in (lambda: awq.paged_plan(i, i, table, i, 16, 2), lambda: awq.kv_append(q, q, cache, cache, slots),
                 lambda: awq.tree_attention(q, cache, cache, table, i, i, 1.0, 2, 0), lambda: awq.process_logits(x)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_package_imports_with_a_torch_that_has_no_package_metadata():
    """A torch of one's own build on the path, say; and the module's name tells torch and Python apart."""
    code = """
import importlib.metadata, sys
def missing(name, *_):
    raise importlib.metadata.PackageNotFoundError(name)
import torch
importlib.metadata.version = missing
from bit_weight_quantized_awq_gb300 import _binding, build
assert build.STEP_MODULE == _binding.STEP_PATH
assert torch.__version__ in _binding.STEP_PATH and sys.implementation.cache_tag in _binding.STEP_PATH
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
