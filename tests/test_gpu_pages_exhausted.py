"""GPU tests of a cache that has run out, with the list that free_pages gives: as long as the cache, -1 after the
last free block. Where a plan or a fork comes to such an entry, there is no free block left."""
import numpy as np
import pytest
import torch

import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import Status

pytestmark = pytest.mark.gpu

PAGE = 16


@pytest.fixture(autouse=True)
def _status(gpu):
    """Every test starts and ends with a clean device status."""
    awq.awq_last_device_status(None)
    yield
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


def i32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


def cache(left):
    """Two rows of 20 tokens in a cache that has `left` more blocks, and its free list."""
    table, lens = i32([[0, 1, -1, -1], [2, 3, -1, -1]]), i32([20, 20])
    free = awq.free_pages(table, lens, PAGE, 4 + left)
    assert free.counts.tolist() == [left, 4] and free.free_blocks.numel() == 4 + left
    return table, lens, free.free_blocks


@pytest.mark.parametrize("left", [0, 1, 2])
def test_a_fork_finds_no_free_block(left):
    table, lens, free = cache(left)
    f = awq.fork_pages(table, lens, i32([0, 0, 1, 1]), free, PAGE)            # two copies
    assert awq.awq_last_device_status(None) == (Status.OK if left == 2 else Status.ERR_TOO_LARGE)
    got = [4 + i if i < left else -1 for i in range(2)]
    assert f.block_table[:, 1].tolist() == [1, got[0], 3, got[1]] and f.block_table[:, 0].tolist() == [0, 0, 2, 2]
    assert f.dst.tolist() == got + [-1, -1] and f.src.tolist() == [1 if left > 0 else -1, 3 if left > 1 else -1, -1, -1]
    assert f.count.tolist() == [2] and f.lens.tolist() == [20] * 4


@pytest.mark.parametrize("start", [0, 1, 2])
def test_a_fork_finds_none_behind_what_a_plan_took(start):
    table, lens, free = cache(3)
    f = awq.fork_pages(table, lens, i32([0, 0, 1, 1]), free, PAGE, free_start=i32([start]))
    assert awq.awq_last_device_status(None) == (Status.OK if start < 2 else Status.ERR_TOO_LARGE)
    assert f.dst[:2].tolist() == [4 + start, 5 + start if start < 2 else -1]


@pytest.mark.parametrize("left", [0, 1, 2])
def test_a_plan_finds_no_free_block(left):
    table, lens, free = cache(left)
    plan = awq.paged_plan(lens, i32([13, 13]), table, free, PAGE, 26)         # the last token of each in a new block
    assert awq.awq_last_device_status(None) == (Status.OK if left == 2 else Status.ERR_TOO_LARGE)
    slots = plan.slot_map.tolist()
    assert slots[:12] == list(range(20, 32)) and slots[13:25] == list(range(52, 64))
    assert [slots[12], slots[25]] == [(4 + i) * PAGE if i < left else -1 for i in range(2)]
    assert table[:, 2].tolist() == [4 + i if i < left else -1 for i in range(2)]
    assert plan.counts.tolist() == [26, 2]


@pytest.mark.parametrize("bad", [-2, -2 ** 31])
def test_other_negative_entries_are_bad_input(bad):
    table, lens, _ = cache(2)
    f = awq.fork_pages(table, lens, i32([0, 0]), i32([bad]), PAGE)
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    assert f.block_table.tolist()[1] == [0, -1, -1, -1] and f.dst.tolist() == f.src.tolist() == [-1, -1]
    plan = awq.paged_plan(lens, i32([13, 0]), table, i32([bad]), PAGE, 13)
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    assert plan.slot_map.tolist() == list(range(20, 32)) + [-1]
