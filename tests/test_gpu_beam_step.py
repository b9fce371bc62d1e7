"""A step's rotary positions, beam search and pages as they run together: captured into a graph and
replayed, on streams, several calls at once. Results are those of the same calls one by one."""
import numpy as np
import pytest
import torch

import beam_reference as ref
import bit_weight_quantized_awq_gb300 as awq
from bit_weight_quantized_awq_gb300 import Status

pytestmark = pytest.mark.gpu

PAGE, HEADS, KV, DIM, V = 16, 8, 2, 64, 5003


@pytest.fixture(autouse=True)
def _status(gpu):
    """Every test starts and ends with a clean device status."""
    awq.awq_last_device_status(None)
    yield
    torch.cuda.synchronize()
    assert awq.awq_last_device_status(None) == Status.OK


class State:
    """B requests of W beams, a few tokens in, each beam with pages of its own behind shared ones."""

    def __init__(self, B, W, seed):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        lens = np.repeat(rng.integers(1, 70, B), W)
        rows, at = [], 0
        for b in range(B):
            n = int(lens[b * W])
            shared, have = n // 2 // PAGE, -(-n // PAGE)
            for w in range(W):
                rows.append(list(range(at, at + shared)) + list(range(at + shared + w * (have - shared),
                                                                      at + shared + (w + 1) * (have - shared))))
            at += shared + W * (have - shared)
        self.blocks = at + 3 * B * W
        perm = rng.permutation(self.blocks)
        table = np.full((B * W, 8), -1)
        for r, row in enumerate(rows):
            table[r, :len(row)] = perm[row]
        i32 = lambda v: torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")  # noqa: E731
        self.table, self.lens, self.ones = i32(table), i32(lens), i32(np.ones(B * W))
        self.caches = [torch.randn((self.blocks, PAGE, KV, DIM), device="cuda", generator=gen).half() for _ in range(4)]
        self.qkv = torch.randn((B * W, HEADS + 2 * KV, DIM), device="cuda", generator=gen).half()
        self.logits = torch.randn((B * W, V), device="cuda", generator=gen).half()
        self.scores = -torch.rand((B, W), device="cuda", generator=gen)
        self.history = torch.randint(V, (B * W, 11), device="cuda", generator=gen, dtype=torch.int32)
        self.inv_freq = (10000.0 ** (-torch.arange(DIM // 2) / (DIM // 2))).float().cuda()
        self.ends = i32([3, 4])
        self.W = W

    def run(self):
        free = awq.free_pages(self.table, self.lens, PAGE, self.blocks)
        plan = awq.paged_plan(self.lens, self.ones, self.table, free.free_blocks, PAGE, self.lens.numel())
        outs = []
        for k_cache, v_cache in (self.caches[:2], self.caches[2:]):
            q = awq.rotary_append(self.qkv[:, :HEADS], self.qkv[:, HEADS:HEADS + KV], self.qkv[:, HEADS + KV:], plan.positions,
                                  self.inv_freq, k_cache, v_cache, plan.slot_map)
            outs.append(awq.tree_attention(q, k_cache, v_cache, self.table, self.lens, plan.cu_new, DIM ** -0.5, 1, 128))
        step = awq.beam_select(self.logits, self.scores, self.W, end_tokens=self.ends)
        parents = step.parents.view(-1)
        history, = awq.reorder_states([self.history], parents)
        f = awq.fork_pages(self.table, self.lens + 1, parents, free.free_blocks, PAGE, free_start=plan.counts[1:])
        awq.copy_pages(self.caches, f.src, f.dst, f.tokens, f.count)
        c = awq.compact_pages(f.block_table, f.lens, PAGE, self.blocks)
        awq.copy_pages(self.caches, c.src, c.dst, count=c.count)
        return [*outs, *step, history, *f, *c, *free]

    def tensors(self):
        return [self.table, self.lens, *self.caches, self.qkv, self.logits, self.scores, self.history]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def content(s, table, lens):
    """What each row's pages hold, in all caches."""
    table, lens = table.cpu().numpy(), lens.tolist()
    return [[c[table[r, :-(-n // PAGE)]].flatten(0, 1)[:n].clone() for c in s.caches] for r, n in enumerate(lens)]


def test_a_step_keeps_what_the_beams_hold():
    s = State(5, 4, 0)
    outs = s.run()
    parents, table, lens, new_table = outs[3].view(-1), outs[9], outs[10], outs[15]
    # the beams' pages before fork and compaction are those of the same state without them
    t = State(5, 4, 0)
    free = awq.free_pages(t.table, t.lens, PAGE, t.blocks)
    plan = awq.paged_plan(t.lens, t.ones, t.table, free.free_blocks, PAGE, t.lens.numel())
    for k_cache, v_cache in (t.caches[:2], t.caches[2:]):
        awq.rotary_append(t.qkv[:, :HEADS], t.qkv[:, HEADS:HEADS + KV], t.qkv[:, HEADS + KV:], plan.positions, t.inv_freq,
                          k_cache, v_cache, plan.slot_map)
    before, after = content(t, t.table, t.lens + 1), content(s, new_table, lens)
    assert table.shape == s.table.shape
    for r, p in enumerate(parents.tolist()):
        assert same(after[r], before[p])
    used = ref.used(new_table.cpu().numpy(), lens.tolist(), PAGE, s.blocks)
    assert used[:used.sum()].all()
    # partly filled pages are in one row only
    last = [int(new_table[r, n // PAGE]) for r, n in enumerate(lens.tolist()) if n % PAGE]
    assert len(set(last)) == len(last)


def test_a_step_is_captured_and_replayed():
    """With the inputs of its capture, with others, and with the first again."""
    s, other = State(7, 3, 1), State(7, 3, 1)
    other.logits, other.scores = torch.randn_like(other.logits), other.scores.flip(0).contiguous()
    other.qkv = other.qkv.flip(0).contiguous()
    inputs, want = [], []
    for state in (s, other):
        inputs.append([x.clone() for x in state.tensors()])
        want.append([[x.clone() for x in state.run()], [x.clone() for x in state.caches]])
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        awq.awq_reserve_tree_attention(DIM, stream.cuda_stream)
        with torch.cuda.graph(graph, stream=stream):
            outs = s.run()
    for i in (0, 1, 0):
        for x, y in zip(s.tensors(), inputs[i]):
            x.copy_(y)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(outs, want[i][0]) and same(s.caches, want[i][1])


def test_calls_on_several_streams_at_once():
    states = [State(6, 4, i) for i in range(4)]
    keep = [[x.clone() for x in s.tensors()] for s in states]
    want = [[x.clone() for x in s.run()] for s in states]
    for s, k in zip(states, keep):
        for x, y in zip(s.tensors(), k):
            x.copy_(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = []
    for s, stream in zip(states, streams):
        with torch.cuda.stream(stream):
            got.append(s.run())
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert same(g, w)


def test_two_graphs_replayed_at_once():
    """Workspaces are the calls' own: no two captures share one."""
    states = [State(4, 8, i) for i in range(2)]
    keep = [[x.clone() for x in s.tensors()] for s in states]
    want, graphs, streams, outs = [], [], [torch.cuda.Stream() for _ in states], []
    for s, k, stream in zip(states, keep, streams):
        want.append([x.clone() for x in s.run()])
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            awq.awq_reserve_tree_attention(DIM, stream.cuda_stream)
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                outs.append(s.run())
        for x, y in zip(s.tensors(), k):
            x.copy_(y)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, k, stream, graph in zip(states, keep, streams, graphs):
            with torch.cuda.stream(stream):
                for x, y in zip(s.tensors(), k):
                    x.copy_(y)
                graph.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert same(o, w)
