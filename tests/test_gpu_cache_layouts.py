"""GPU tests of copy_pages with caches whose layouts are the same though their strides are written differently: the
stride of an axis with one entry says nothing."""
import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import Status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("blocks,heads", [(9, 1), (1, 2), (1, 1)])
def test_strides_of_single_entries_do_not_matter(gpu, blocks, heads):
    shape = (blocks, 16, heads, 64)
    plain = torch.randn(shape, device="cuda").half()
    # one head of a heads-first cache, one block of a wider allocation
    other = torch.empty(0, dtype=torch.float16, device="cuda").set_(
        torch.randn(shape, device="cuda").half().untyped_storage(), 0, shape,
        (16 * heads * 64 if blocks > 1 else 99968, heads * 64, 16 * 64 if heads == 1 else 64, 1))
    assert plain.stride() != other.stride()
    pairs = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([blocks - 1, -1], [0, 0])]
    want = [c.clone() for c in (plain, other)]
    for c in want:
        c[0] = c[blocks - 1].clone()
    awq.copy_pages([plain, other], *pairs)
    assert all(torch.equal(a, b) for a, b in zip((plain, other), want))
    assert gpu.awq_last_device_status(None) == Status.OK


def test_other_layouts_are_refused(gpu):
    a = torch.zeros((4, 16, 2, 64), device="cuda").half()
    pairs = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([1], [0])]
    for b in (torch.zeros((4, 2, 16, 64), device="cuda").half().transpose(1, 2), a.bfloat16(), a[:3],
              torch.zeros((4, 16, 2, 72), device="cuda").half()[..., :64], a.cpu()):
        with pytest.raises(ValueError):
            awq.copy_pages([a, b], *pairs)
