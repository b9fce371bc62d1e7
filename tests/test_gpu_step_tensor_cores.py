"""The tensor-core kernel of tree_attention, taken because the bounds allow a long cache,
in the forms in which it differs from the few-row kernel: its own products, tensor maps
and pieces. Tolerances as in test_gpu_step.py."""
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


@pytest.mark.parametrize("heads,kv_heads,new", [(8, 8, 26), (16, 2, 13), (16, 2, 64)])
@pytest.mark.parametrize("dim", [64, 128])
def test_every_call_gives_the_same_bits(heads, kv_heads, new, dim):
    """S of a tile is written over the weights of the tile before: only after their product
    with V. Streams, halves and CTAs meet in another order from call to call; the sums do not."""
    s = Step([3000, 700, 1500, 90], [new, new // 2, new, 1], heads, kv_heads, dim, 32, torch.float16, "tree", seed=new)
    out, lse = s.run(max_context=LONG)
    s.check(out, lse)
    args = (s.q.cuda(), s.k.cuda(), s.v.cuda(), i32(s.table), i32(s.ctx), i32(s.cu))
    mask = s.mask.cuda()
    for _ in range(200):
        assert torch.equal(awq.tree_attention(*args, s.scale, new, LONG, tree_mask=mask), out)
