"""Results of a step that a caller keeps hold no workspace: their storage is the results alone."""
import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import Status

pytestmark = pytest.mark.gpu


def storage_of(results):
    """Bytes of the storages behind a tuple of tensors, and of the tensors."""
    tensors = [t for t in results if t is not None]
    storages = {t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in tensors}
    return sum(storages.values()), sum(t.numel() * t.element_size() for t in tensors)


def test_results_keep_no_workspace(gpu):
    logits = torch.randn((16 * 4, 50000), device="cuda").half()
    before = -torch.rand((16, 4), device="cuda")
    ends = torch.tensor([3], dtype=torch.int32, device="cuda")
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(8, 8)
    lens = torch.full((8,), 100, dtype=torch.int32, device="cuda")
    for results in (awq.beam_select(logits, before, 4), awq.beam_select(logits, before, 4, end_tokens=ends),
                    awq.free_pages(table, lens, 16, 100000), awq.free_pages(table, lens, 16, 1000000),
                    awq.compact_pages(table, lens, 16, 100000), awq.compact_pages(table, lens, 16, 1000000)):
        held, needed = storage_of(results)
        assert held == needed
    assert gpu.awq_last_device_status(None) == Status.OK


def test_calls_one_after_the_other_share_no_results(gpu):
    """The workspace of one call may be the memory of the next one's; results stay as they are."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    cases = [(torch.randn((8, 30000 + 7 * i), device="cuda", generator=gen), -torch.rand((2, 4), device="cuda", generator=gen))
             for i in range(6)]
    tables = [(torch.randperm(400, device="cuda", generator=gen).int()[:64].view(8, 8),
               torch.randint(0, 129, (8,), device="cuda", generator=gen, dtype=torch.int32)) for _ in range(6)]

    def every():
        for (x, s), (t, n) in zip(cases, tables):
            yield awq.beam_select(x, s, 4)[:3]
            yield awq.free_pages(t, n, 16, 400)
            yield awq.compact_pages(t, n, 16, 400000)
    together = list(every())
    torch.cuda.synchronize()
    for a, b in zip(together, every()):
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert gpu.awq_last_device_status(None) == Status.OK
