"""What the decoding step's functions refuse before anything runs: wrong types, devices,
shapes, strides and lengths of tensors. The library's own refusals are in
test_step_boundary.py, what only the device can see in test_gpu_step.py."""
import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import AWQError

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(gpu):
    pass


def ints(*shape, value=1):
    return torch.full(shape, value, dtype=torch.int32, device="cuda")


def halves(*shape):
    return torch.zeros(shape, dtype=torch.float16, device="cuda")


def plan_arguments():
    return dict(context_lens=ints(3), new_lens=ints(3), block_table=ints(3, 4, value=0), free_blocks=ints(8),
                block_size=16, max_tokens=6, parents=ints(6, value=-1), mask_words=1)


def append_arguments():
    return dict(k=halves(5, 2, 64), v=halves(5, 2, 64), k_cache=halves(4, 16, 2, 64), v_cache=halves(4, 16, 2, 64),
                slot_map=torch.arange(5, device="cuda"))


def attention_arguments():
    return dict(q=halves(3, 4, 64), k_cache=halves(4, 16, 2, 64), v_cache=halves(4, 16, 2, 64), block_table=ints(2, 2),
                context_lens=ints(2), cu_new=torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda"), scale=0.125,
                max_new=2, max_context=1, tree_mask=ints(3, 1, value=3), out=halves(3, 4, 64),
                lse=torch.zeros((3, 4), device="cuda"))


def logits_arguments():
    return dict(logits=halves(4, 100), row_request=ints(4, value=0), history=ints(10), history_offsets=ints(3, value=0),
                prompt_lens=ints(2), repetition=torch.ones(2, device="cuda"), frequency=torch.ones(2, device="cuda"),
                presence=torch.ones(2, device="cuda"), draft_tokens=ints(4), cu_new=ints(3, value=0),
                tree_mask=ints(4, 1), bias_tokens=ints(5), bias_values=torch.ones(5, device="cuda"),
                bias_offsets=ints(3, value=0), grammar_mask=ints(4, 4, value=-1), grammar_rows=ints(4, value=0),
                out=halves(4, 100))


ALL = [(awq.paged_plan, plan_arguments), (awq.kv_append, append_arguments), (awq.tree_attention, attention_arguments),
       (awq.process_logits, logits_arguments)]


@pytest.mark.parametrize("call,arguments", ALL)
def test_arguments_as_they_should_be_are_taken(call, arguments):
    call(**arguments())
    torch.cuda.synchronize()
    awq.awq_last_device_status(None)


@pytest.mark.parametrize("call,arguments", ALL)
def test_tensors_of_another_type_device_or_length(call, arguments):
    for name, good in arguments().items():
        if not isinstance(good, torch.Tensor):
            continue
        wrong = [good.cpu(), good.double(), good.reshape(-1)[:-1] if good.dim() == 1 else good[..., None]]
        if name in ("free_blocks", "history"):         # of any length
            wrong.pop()
        for bad in wrong:
            kw = arguments()
            kw[name] = bad
            with pytest.raises(ValueError):
                call(**kw)
        kw = arguments()
        kw[name] = [1, 2]
        with pytest.raises(TypeError):
            call(**kw)


@pytest.mark.parametrize("call,arguments", ALL)
def test_whole_numbers_are_whole_numbers(call, arguments):
    for name, good in arguments().items():
        if isinstance(good, int):
            with pytest.raises(TypeError):
                call(**dict(arguments(), **{name: 1.5}))


@pytest.mark.parametrize("call,arguments,name,bad", [
    (awq.paged_plan, plan_arguments, "context_lens", lambda t: ints(6)[::2]),
    (awq.paged_plan, plan_arguments, "block_table", lambda t: ints(4, 3).T),
    (awq.paged_plan, plan_arguments, "max_tokens", lambda t: -1),
    (awq.paged_plan, plan_arguments, "mask_words", lambda t: -1),
    (awq.kv_append, append_arguments, "k", lambda t: halves(5, 64, 2).transpose(1, 2)),
    (awq.kv_append, append_arguments, "k", lambda t: halves(5, 3, 64)),
    (awq.kv_append, append_arguments, "v", lambda t: t.bfloat16()),
    (awq.kv_append, append_arguments, "v_cache", lambda t: halves(4, 16, 64, 2).transpose(2, 3)),
    (awq.kv_append, append_arguments, "v_cache", lambda t: halves(4, 32, 2, 64)),
    (awq.tree_attention, attention_arguments, "q", lambda t: halves(3, 64, 4).transpose(1, 2)),
    (awq.tree_attention, attention_arguments, "q", lambda t: halves(3, 4, 72)),
    (awq.tree_attention, attention_arguments, "block_table", lambda t: ints(3, 2)),
    (awq.tree_attention, attention_arguments, "tree_mask", lambda t: ints(3, 0)),
    (awq.tree_attention, attention_arguments, "out", lambda t: halves(3, 64, 4).transpose(1, 2)),
    (awq.tree_attention, attention_arguments, "out", lambda t: halves(4, 3, 64)),
    (awq.tree_attention, attention_arguments, "lse", lambda t: torch.zeros((4, 3), device="cuda")),
    (awq.process_logits, logits_arguments, "logits", lambda t: halves(100, 4).T),
    (awq.process_logits, logits_arguments, "out", lambda t: halves(100, 4).T),
    (awq.process_logits, logits_arguments, "tree_mask", lambda t: ints(5, 1)),
    (awq.process_logits, logits_arguments, "grammar_mask", lambda t: ints(4, 3)),
    (awq.process_logits, logits_arguments, "history_offsets", lambda t: None),
    (awq.process_logits, logits_arguments, "bias_values", lambda t: None),
    (awq.process_logits, logits_arguments, "bias_offsets", lambda t: None),
    (awq.process_logits, logits_arguments, "cu_new", lambda t: None)])
def test_shapes_strides_and_what_belongs_together(call, arguments, name, bad):
    kw = arguments()
    kw[name] = bad(kw[name])
    with pytest.raises(ValueError):
        call(**kw)


def test_statuses_of_the_library_become_its_error():
    kw = plan_arguments()
    with pytest.raises(AWQError, match="awq_paged_plan"):
        awq.paged_plan(**dict(kw, block_size=24))
    kw = append_arguments()
    kw["k"] = torch.zeros(5 * 2 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(5, 2, 64)     # not on 16 bytes
    with pytest.raises(AWQError, match="awq_kv_append"):
        awq.kv_append(**kw)
    with pytest.raises(AWQError, match="awq_tree_attention"):
        awq.tree_attention(**dict(attention_arguments(), max_new=-1))
    kw = logits_arguments()
    kw["out"] = torch.zeros((4, 200), dtype=torch.float16, device="cuda")[:, :100]
    awq.process_logits(**kw)                           # another stride is fine, unless in place
    with pytest.raises(AWQError, match="awq_process_logits"):
        awq.process_logits(kw["logits"], bias_values=kw["bias_values"])
    torch.cuda.synchronize()
    awq.awq_last_device_status(None)


@pytest.mark.parametrize("name,bad", [("max_tokens", 2 ** 30 + 1), ("max_tokens", 2 ** 40), ("max_tokens", 2 ** 61),
                                      ("max_tokens", 2 ** 62), ("mask_words", 1025), ("mask_words", 2 ** 50),
                                      ("mask_words", 2 ** 62)])
def test_sizes_that_no_plan_has_are_refused_before_memory_is_asked_for(name, bad):
    kw = dict(plan_arguments(), parents=None)
    kw[name] = bad
    with pytest.raises(ValueError, match=name):
        awq.paged_plan(**kw)
