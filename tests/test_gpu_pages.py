"""GPU tests of fork_pages, copy_pages, free_pages and compact_pages against references on the
CPU. Everything here is whole numbers and copies: compared for equality."""
import numpy as np
import pytest
import torch

import beam_reference as ref
import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import AWQError, Status

pytestmark = pytest.mark.gpu

FP16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _status(gpu):
    """Every test starts and ends with a clean device status."""
    awq.awq_last_device_status(None)
    yield
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


def i32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device="cuda")


def tables(rng, lens, page, spare=5, extra=2):
    """(table, blocks that no row has, blocks in all)."""
    have = [-(-n // page) for n in lens]
    total = sum(have) + spare
    perm = rng.permutation(total)
    table = np.full((len(lens), max(have + [0]) + extra), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, perm[at:], total


# ---------------------------------------------------------------- fork

def check_fork(table, lens, parents, free, page, start=None):
    want, want_lens, pairs = ref.fork(table, lens, parents, free, page, start or 0)
    f = awq.fork_pages(i32(table), i32(lens), i32(parents), i32(free), page, free_start=None if start is None else i32([start]))
    assert f.block_table.tolist() == want.tolist() and f.lens.tolist() == [max(n, 0) for n in want_lens]
    assert f.count.tolist() == [len(pairs)]
    for got, i in ((f.src, 0), (f.dst, 1), (f.tokens, 2)):
        assert got.tolist() == [p[i] for p in pairs] + [-1] * (len(parents) - len(pairs))
    return f


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("rows,out", [(1, 1), (1, 32), (8, 8), (40, 13), (600, 1500), (3, 0)])
def test_fork_matches_the_reference(page, rows, out):
    rng = np.random.default_rng(rows + out)
    lens = rng.integers(0, 5 * page, rows)
    lens[rng.random(rows) < 0.2] = 2 * page         # full last pages
    table, free, _ = tables(rng, lens, page, spare=out + 9)
    parents = rng.integers(-1, rows, out)
    check_fork(table, lens, parents, free, page)
    check_fork(table, lens, parents, free, page, start=4)


def test_fork_of_wide_tables_and_the_most_rows():
    rng = np.random.default_rng(0)
    lens = [16 * 5000 + 3, 16 * 2048, 16 * 2047 + 1, 7]
    table, free, _ = tables(rng, lens, 16)
    check_fork(table, lens, [0, 0, 1, 1, 2, 2, 3], free, 16)
    lens = rng.integers(0, 64, 16384)
    table, free, _ = tables(rng, lens, 16, spare=16384)
    check_fork(table, lens, rng.integers(0, 16384, 16384), free, 16)


def test_fork_reads_views_of_tables():
    lens = [20, 33]
    wide = torch.full((2, 9), 77, dtype=torch.int32, device="cuda")
    wide[:, 2:5] = i32([[4, 9, -1], [1, 0, 6]])
    f = awq.fork_pages(wide[:, 2:5], i32(lens), i32([1, 1, 0]), i32([8, 7]), 16)
    assert f.block_table.tolist() == [[1, 0, 6], [1, 0, 8], [4, 9, -1]] and f.lens.tolist() == [33, 33, 20]
    assert (f.src.tolist(), f.dst.tolist(), f.tokens.tolist()) == ([6, -1, -1], [8, -1, -1], [1, -1, -1])


def test_fork_reports_what_does_not_fit():
    table, free = i32([[0, 1], [2, 3]]), i32([9])
    f = awq.fork_pages(table, i32([20, 20]), i32([0, 0, 1, 1]), free, 16)         # one block for two copies
    assert awq.awq_last_device_status(None) == Status.ERR_TOO_LARGE
    assert f.block_table.tolist() == [[0, 1], [0, 9], [2, 3], [2, -1]] and f.count.tolist() == [2]
    assert f.src.tolist() == [1, -1, -1, -1] and f.dst.tolist() == [9, -1, -1, -1]
    f = awq.fork_pages(table, i32([40, -3]), i32([0, 0, 1]), free, 16)            # longer than the table, negative
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    assert f.block_table.tolist() == [[0, 1], [0, 1], [-1, -1]] and f.count.tolist() == [0] and f.lens.tolist() == [40, 40, 0]
    f = awq.fork_pages(table, i32([20, 20]), i32([2, -2, 1]), free, 16)           # no such parents
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    assert f.block_table.tolist() == [[-1, -1], [-1, -1], [2, 3]] and f.lens.tolist() == [0, 0, 20]
    f = awq.fork_pages(table, i32([20, 20]), i32([0, 0]), free, 16, free_start=i32([-5]))
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG and f.dst.tolist() == [9, -1]
    f = awq.fork_pages(table, i32([20, 20]), i32([0, 0]), free, 16, free_start=i32([2 ** 31 - 1]))
    assert awq.awq_last_device_status(None) == Status.ERR_TOO_LARGE and f.dst.tolist() == [-1, -1]
    f = awq.fork_pages(i32([[0, -1]]), i32([20]), i32([0, 0]), free, 16)          # a page that is not there
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG and f.src.tolist() == [-1, -1]


# ---------------------------------------------------------------- copy

def caches_of(kind, n, blocks, page, heads, dim, dtype):
    if kind == "heads_first":
        return [torch.randn((blocks, heads, page, dim), device="cuda").to(dtype).transpose(1, 2) for _ in range(n)]
    if kind == "together":       # keys and values of a block beside each other
        both = [torch.randn((blocks, 2, page, heads, dim), device="cuda").to(dtype) for _ in range((n + 1) // 2)]
        return [c for kv in both for c in (kv[:, 0], kv[:, 1])][:n]
    if kind == "padded":         # rows of a wider array
        return [torch.randn((blocks, page, heads, dim + 8), device="cuda").to(dtype)[..., :dim] for _ in range(n)]
    return [torch.randn((blocks, page, heads, dim), device="cuda").to(dtype) for _ in range(n)]


@pytest.mark.parametrize("kind", ["plain", "heads_first", "together", "padded"])
@pytest.mark.parametrize("n,page,heads,dim,dtype", [(1, 16, 1, 8, FP16), (4, 16, 8, 128, BF16), (3, 64, 3, 80, FP16), (2, 1024, 2, 64, BF16)])
def test_pages_are_copied(kind, n, page, heads, dim, dtype):
    blocks = 23
    rng = np.random.default_rng(page + heads)
    caches = caches_of(kind, n, blocks, page, heads, dim, dtype)
    perm = rng.permutation(blocks)
    src, dst = np.append(perm[:9], [3, -1, 5]), np.append(perm[9:18], [-1, 4, 5])       # -1: none; 5: itself
    src[2] = src[1]                                                                     # one block to several
    tokens = rng.integers(0, page + 1, 12)
    tokens[0], tokens[1] = 0, page
    for given, count in ((None, None), (tokens, None), (tokens, 4), (None, 0), (tokens, 99), (None, -1)):
        before = [c.clone() for c in caches]
        awq.copy_pages(caches, i32(src), i32(dst), tokens=None if given is None else i32(given),
                       count=None if count is None else i32([count]))
        for i, (s, d) in enumerate(zip(src, dst)):
            if s < 0 or d < 0 or (count is not None and i >= count):
                continue
            t = page if given is None else given[i]
            for b in before:
                b[d, :t] = b[s, :t].clone()
        for c, b in zip(caches, before):
            assert torch.equal(c, b)


def test_copies_in_more_caches_than_a_launch_takes():
    caches = caches_of("plain", 300, 3, 16, 1, 8, FP16)
    before = [c.clone() for c in caches]
    awq.copy_pages(caches, i32([2]), i32([0]))
    for c, b in zip(caches, before):
        assert torch.equal(c[0], b[2]) and torch.equal(c[1:], b[1:])


def test_blocks_behind_the_first_four_gigabytes():
    cache = torch.zeros((40000, 64, 8, 128), device="cuda", dtype=FP16)      # 5.2 GB
    cache[39999] = 3
    awq.copy_pages([cache], i32([39999]), i32([39997]), tokens=i32([63]))
    assert (cache[39997, :63] == 3).all() and (cache[39997, 63] == 0).all() and (cache[39998] == 0).all()


@pytest.mark.parametrize("kind", ["plain", "heads_first", "together"])
@pytest.mark.parametrize("page,heads,dim", [(64, 8, 128), (32, 3, 136), (1024, 1, 64), (16, 40, 80)])
def test_many_bytes_go_in_bulk(kind, page, heads, dim):
    """Long runs, many pages: parts of pages, none of them, and counts that say less than the lists."""
    blocks = 2 * (1 + 4_000_000 // (page * heads * dim)) + 5
    rng = np.random.default_rng(page)
    caches = caches_of(kind, 5, blocks, page, heads, dim, BF16)
    perm = rng.permutation(blocks)
    n = (blocks - 5) // 2
    src, dst, tokens = perm[:n].copy(), perm[n:2 * n].copy(), rng.integers(0, page + 1, n)
    tokens[:3] = 0, page, 1
    src[n // 2], dst[n // 3] = -1, -1
    dst[n // 4] = src[n // 4]
    for given, count in ((None, None), (tokens, n - 2), (tokens, 0)):
        want = [c.clone() for c in caches]
        awq.copy_pages(caches, i32(src), i32(dst), tokens=None if given is None else i32(given),
                       count=None if count is None else i32([count]))
        good = (src >= 0) & (dst >= 0) & (np.arange(n) < (n if count is None else count))
        t = np.full(n, page) if given is None else given
        kept = torch.from_numpy(np.arange(page) < t[good][:, None]).cuda()[:, :, None, None]
        s, d = torch.from_numpy(src[good]).cuda(), torch.from_numpy(dst[good]).cuda()
        for w in want:
            w[d] = torch.where(kept, w[s], w[d])
        for c, w in zip(caches, want):
            assert torch.equal(c, w)
    bad = src.copy()
    bad[0], bad[1] = blocks, -7
    want = [c.clone() for c in caches]
    long = tokens.copy()
    long[2] = page + 1
    awq.copy_pages(caches, i32(bad[:3]).repeat(n), i32(dst[:3]).repeat(n), tokens=i32(long[:3]).repeat(n), count=i32([3]))
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    for c, w in zip(caches, want):
        if dst[2] >= 0 and bad[2] >= 0:
            w[int(dst[2])] = w[int(bad[2])]
        assert torch.equal(c, w)


@pytest.mark.parametrize("kind", ["plain", "heads_first", "together"])
@pytest.mark.parametrize("page,dim", [(16, 32), (16, 40), (16, 24), (64, 16)])
def test_small_pages_in_bulk(kind, page, dim):
    """Pages of one run from a KB on (and one below), of which few tokens are copied."""
    blocks, n = 8000, 3500
    rng = np.random.default_rng(dim)
    caches = caches_of(kind, 3, blocks, page, 1, dim, FP16)
    perm, tokens = rng.permutation(blocks), rng.integers(0, page + 1, n)
    src, dst = perm[:n], perm[n:2 * n]
    before = [c.clone() for c in caches]
    awq.copy_pages(caches, i32(src), i32(dst), tokens=i32(tokens), count=i32([n - 100]))
    s, d, t = (torch.from_numpy(x[:n - 100]).cuda().long() for x in (src, dst, tokens))
    keep = (torch.arange(page, device="cuda")[None] >= t[:, None])[..., None, None]
    for c, b in zip(caches, before):
        b[d] = torch.where(keep, b[d], b[s])
        assert torch.equal(c, b)


def test_bad_pairs_are_skipped_and_reported():
    cache = torch.randn((4, 16, 1, 8), device="cuda").half()
    before = cache.clone()
    awq.copy_pages([cache], i32([0, 4, -2]), i32([4, 1, 2]))
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG and torch.equal(cache, before)
    awq.copy_pages([cache], i32([0, 1]), i32([2, 3]), tokens=i32([17, -1]))
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    assert torch.equal(cache[2], before[0]) and torch.equal(cache[3], before[3])


# ---------------------------------------------------------------- free and compact

def check_pages(table, lens, page, blocks, held=None):
    held_list = [] if held is None else held
    args = (i32(table), i32(lens), page, blocks, None if held is None else i32(held))
    used = ref.used(table, lens, page, blocks, held_list)
    f = awq.free_pages(*args)
    free = np.flatnonzero(~used)
    assert f.counts.tolist() == [len(free), blocks - len(free)]
    assert np.array_equal(f.free_blocks.cpu().numpy(), np.append(free, np.full(blocks - len(free), -1)))
    want, to, pairs = ref.compact(table, lens, page, blocks, held_list)
    c = awq.compact_pages(*args)
    assert np.array_equal(c.block_table.cpu().numpy(), want) and np.array_equal(c.block_map.cpu().numpy(), to)
    assert c.count.tolist() == [len(pairs)]
    for got, i in ((c.src, 0), (c.dst, 1)):
        assert got.tolist() == [p[i] for p in pairs] + [-1] * (blocks // 2 - len(pairs))


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("rows,longest,spare", [(1, 1, 0), (1, 1, 1), (3, 60, 0), (5, 400, 7), (64, 3000, 500), (700, 100, 64),
                                                (2, 20000, 100000)])
def test_free_and_compact_match_the_reference(page, rows, longest, spare):
    rng = np.random.default_rng(rows + longest)
    lens = rng.integers(0, longest + 1, rows)
    lens[0] = longest
    table, free, blocks = tables(rng, lens, page, spare)
    check_pages(table, lens, page, blocks)
    if rows > 2:
        table[1] = table[0]                          # rows that share their pages
        lens[1] = lens[0] // 2
        lens[2] = 0                                  # a request that has ended
        check_pages(table, lens, page, blocks, held=np.append(free[:5], [-1, table[0, 0]]))


@pytest.mark.parametrize("rows,width", [(255, 3), (257, 128), (300, 65), (700, 64), (5000, 33), (9000, 9), (20000, 8), (30001, 1)])
def test_many_short_rows(rows, width):
    """More rows than warps: several beside each other in one, of all widths that share it."""
    rng = np.random.default_rng(rows)
    have = rng.integers(0, width + 1, rows)
    blocks = int(have.sum()) + 50
    table = np.full((rows, width), -7)
    table[np.arange(width)[None] < have[:, None]] = rng.permutation(blocks)[:have.sum()]
    table[rows // 2], have[rows // 2] = table[0], have[0]               # shared
    check_pages(table, np.maximum(0, have * 16 - 5), 16, blocks)


def test_free_and_compact_at_the_ends():
    check_pages(np.zeros((0, 3), dtype=np.int64), [], 16, 100)                                  # no rows
    check_pages(np.full((2, 3), -1), [0, 0], 16, 1)                                             # nothing used
    check_pages(np.arange(96).reshape(2, 48), [16 * 48, 16 * 48], 16, 96)                       # all used
    check_pages(95 - np.arange(40).reshape(2, 20), [16 * 20, 16 * 20 - 15], 16, 96)             # all at the end
    check_pages(np.array([[63, 31, 32, 95]]), [64], 16, 97, held=[96, 96, 0])


def test_free_and_compact_of_millions_of_blocks():
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 16 * 3000, 900)
    table, _, blocks = tables(rng, lens, 16, spare=2_000_003)
    check_pages(table, lens, 16, blocks)


@pytest.mark.parametrize("rows,longest,spare", [(3000, 16 * 600, 1000), (700, 16 * 2000, 0), (2, 40, 300000), (5000, 16 * 3000, 100)])
def test_many_rows_that_share_many_blocks(rows, longest, spare):
    """More entries than blocks, from a few thousand blocks to millions."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, longest + 1, rows)
    have = -(-lens // 16)
    blocks = max(int(have.sum()) // 9, 1) + spare
    table = rng.integers(0, blocks, (rows, int(have.max()) + 1))
    check_pages(table, lens, 16, blocks)


def test_tables_that_are_views():
    wide = torch.full((3, 10), -9, dtype=torch.int32, device="cuda")
    wide[:, 4:7] = i32([[5, 6, -1], [1, -1, -1], [7, 2, 0]])
    f = awq.free_pages(wide[:, 4:7], i32([32, 1, 33]), 16, 9)
    assert f.free_blocks.tolist() == [3, 4, 8] + [-1] * 6
    c = awq.compact_pages(wide[:, 4:7], i32([32, 1, 33]), 16, 9)
    assert c.block_table.tolist() == [[5, 3, -1], [1, -1, -1], [4, 2, 0]] and c.src.tolist() == [6, 7, -1, -1]


def test_bad_entries_are_skipped_and_reported():
    table = i32([[0, 9], [2, -1]])
    f = awq.free_pages(table, i32([32, 16]), 16, 9)
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG and f.counts.tolist() == [7, 2]
    c = awq.compact_pages(table, i32([32, 32]), 16, 9)
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG
    assert c.block_table.tolist() == [[0, -1], [1, -1]]
    f = awq.free_pages(table, i32([-4, 16]), 16, 9)
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG and f.counts.tolist() == [8, 1]
    f = awq.free_pages(i32([[0, 1]]), i32([1000]), 16, 9)
    assert awq.awq_last_device_status(None) == Status.ERR_TOO_LARGE and f.counts.tolist() == [7, 2]
    f = awq.free_pages(i32([[0, 1]]), i32([16]), 16, 9, held=i32([9, -2, 3]))
    assert awq.awq_last_device_status(None) == Status.ERR_INVALID_ARG and f.counts.tolist() == [7, 2]


def test_compacted_caches_hold_what_they_held():
    rng = np.random.default_rng(4)
    lens = rng.integers(1, 300, 20)
    table, _, blocks = tables(rng, lens, 16, spare=300)
    caches = [torch.randn((blocks, 16, 2, 64), device="cuda").half() for _ in range(4)]
    before = [c.clone() for c in caches]
    c = awq.compact_pages(i32(table), i32(lens), 16, blocks)
    awq.copy_pages(caches, c.src, c.dst, count=c.count)
    new = c.block_table.cpu().numpy()
    assert new.max() == sum(-(-n // 16) for n in lens) - 1
    for cache, old in zip(caches, before):
        for r, n in enumerate(lens):
            have = -(-n // 16)
            assert torch.equal(cache[new[r, :have]], old[table[r, :have]])


# ---------------------------------------------------------------- refusals

def fork_arguments():
    return dict(block_table=i32([[0, 1], [2, 3]]), lens=i32([20, 5]), parents=i32([0, 1]), free_blocks=i32([4]), block_size=16,
                free_start=i32([0]))


def copy_arguments():
    return dict(caches=[torch.zeros((4, 16, 2, 64), device="cuda", dtype=FP16)], src=i32([0]), dst=i32([1]), tokens=i32([3]), count=i32([1]))


def pages_arguments():
    return dict(block_table=i32([[0, 1], [2, 3]]), lens=i32([20, 5]), block_size=16, num_blocks=8, held=i32([5]))


ALL = [(awq.fork_pages, fork_arguments), (awq.copy_pages, copy_arguments), (awq.free_pages, pages_arguments),
       (awq.compact_pages, pages_arguments)]


@pytest.mark.parametrize("call,make", ALL)
def test_arguments_of_another_kind(call, make):
    call(**make())
    for name, good in make().items():
        if isinstance(good, torch.Tensor):
            wrong = [good.cpu(), good.double(), torch.cat([good, good])] if name not in ("parents", "free_blocks", "held", "block_table") \
                else [good.cpu(), good.long()]
            if good.dim() == 1 and name not in ("count", "free_start"):
                wrong.append(torch.cat([good, good, good, good])[::2])       # not contiguous
            for bad in wrong:
                if call is awq.copy_pages and name == "src" and bad is wrong[2]:
                    continue
                with pytest.raises(ValueError):
                    call(**dict(make(), **{name: bad}))
            with pytest.raises(TypeError):
                call(**dict(make(), **{name: [1]}))
        elif isinstance(good, int):
            with pytest.raises(TypeError):
                call(**dict(make(), **{name: 1.5}))


@pytest.mark.parametrize("call,make,name,bad,error", [
    (awq.fork_pages, fork_arguments, "block_size", 24, AWQError), (awq.fork_pages, fork_arguments, "block_table", None, None),
    (awq.free_pages, pages_arguments, "block_size", 8, AWQError), (awq.free_pages, pages_arguments, "num_blocks", 0, ValueError),
    (awq.free_pages, pages_arguments, "num_blocks", 2 ** 28 + 1, ValueError), (awq.compact_pages, pages_arguments, "num_blocks", 2 ** 40, ValueError),
    (awq.compact_pages, pages_arguments, "block_size", 2048, AWQError)])
def test_sizes(call, make, name, bad, error):
    if error is None:
        bad, error = i32([[0, 1]]), ValueError
    with pytest.raises(error):
        call(**dict(make(), **{name: bad}))


def test_fork_refuses_more_rows_than_it_takes():
    with pytest.raises(ValueError):
        awq.fork_pages(**dict(fork_arguments(), parents=torch.zeros(16385, dtype=torch.int32, device="cuda")))


@pytest.mark.parametrize("bad", [
    lambda c: [c.float()], lambda c: [c.cpu()], lambda c: [c, c[:3]], lambda c: [c, c.bfloat16()],
    lambda c: [c, torch.zeros((4, 2, 16, 64), device="cuda", dtype=FP16).transpose(1, 2)], lambda c: [c[0]]])
def test_caches_that_do_not_agree(bad):
    kw = copy_arguments()
    with pytest.raises(ValueError):
        awq.copy_pages(**dict(kw, caches=bad(kw["caches"][0])))
    with pytest.raises(TypeError):
        awq.copy_pages(**dict(kw, caches=5))
    with pytest.raises(TypeError):
        awq.copy_pages(**dict(kw, caches=[5]))
    awq.copy_pages(**dict(kw, caches=[]))
    awq.copy_pages(**dict(kw, caches=tuple(kw["caches"])))
    empty = i32([])
    awq.copy_pages(kw["caches"], empty, empty)
