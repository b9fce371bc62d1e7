"""Beam search with a small decoder of AWQ-quantised layers over a paged cache whose pages the
beams of a request share.

A prompt is filled in once; its row is forked into the first beams. Every step then runs
``paged_plan``, per layer ``rotary_append`` and ``tree_attention`` between the quantised
projections, ``beam_select`` on the logits, and for the beams that go on ``reorder_states``
(their tokens), ``fork_pages`` and ``copy_pages`` (their cache) and ``free_pages`` (the blocks
that nobody needs any more, which the next plan takes from). Lengths, tables and the free list
stay on the GPU: no step waits for the host.

    python examples/beam_decode.py [--steps 12] [--requests 3] [--beams 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_quantized_awq_gb300 as awq  # noqa: E402
from bit_weight_quantized_awq_gb300.synthetic import make_problem  # noqa: E402

HEADS, KV_HEADS, DIM, LAYERS, VOCAB, PAGE = 8, 2, 64, 2, 1024, 16
HIDDEN = HEADS * DIM


def quantised_layer(K: int, N: int, seed: int) -> awq.AWQLinear:
    p = make_problem(1, K, N, 64, bias=False, seed=seed).to("cuda")
    return awq.AWQLinear(4, 64, p.qweight, p.qzeros, p.scales, None)


def norm(x: torch.Tensor) -> torch.Tensor:
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).half()


class Decoder:
    """Weights and the paged caches; the rows' tables and lengths come with each call."""

    def __init__(self, blocks: int, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)
        self.blocks = blocks
        self.embedding = torch.randn((VOCAB, HIDDEN), generator=gen).half().cuda()
        self.layers = [(quantised_layer(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM, seed + 4 * i),
                        quantised_layer(HIDDEN, HIDDEN, seed + 4 * i + 1)) for i in range(LAYERS)]
        self.head = quantised_layer(HIDDEN, VOCAB, seed + 99)
        self.inv_freq = (10000.0 ** (-torch.arange(DIM // 2) / (DIM // 2))).float().cuda()
        self.caches = [torch.zeros((blocks, PAGE, KV_HEADS, DIM), dtype=torch.float16, device="cuda")
                       for _ in range(2 * LAYERS)]

    def step(self, tokens, lens, new_lens, table, free, longest_new: int, longest: int):
        """Logits [tokens, VOCAB] of the rows' new tokens (row by row) and the step's plan."""
        plan = awq.paged_plan(lens, new_lens, table, free, PAGE, tokens.numel())
        x = self.embedding[tokens.long()]
        for i, (qkv, out) in enumerate(self.layers):
            k_cache, v_cache = self.caches[2 * i:2 * i + 2]
            y = qkv(norm(x)).view(-1, HEADS + 2 * KV_HEADS, DIM)
            q = awq.rotary_append(y[:, :HEADS], y[:, HEADS:HEADS + KV_HEADS], y[:, HEADS + KV_HEADS:], plan.positions,
                                  self.inv_freq, k_cache, v_cache, plan.slot_map)
            a = awq.tree_attention(q, k_cache, v_cache, table, lens, plan.cu_new, DIM ** -0.5, longest_new, longest)
            x = x + out(a.view(-1, HIDDEN))
        return self.head(norm(x)), plan

    def fork(self, table, lens, parents, free, start):
        """The rows that continue `parents`: their tables, lengths, and the blocks that are free then."""
        f = awq.fork_pages(table, lens, parents, free, PAGE, free_start=start)
        awq.copy_pages(self.caches, f.src, f.dst, f.tokens, f.count)
        return f.block_table, f.lens, awq.free_pages(f.block_table, f.lens, PAGE, self.blocks).free_blocks


class BeamSearch:
    """The beams of all requests, and the best of those that ended, by score / length ** alpha."""

    def __init__(self, model: Decoder, prompts: list[list[int]], beams: int, ends: list[int], pages: int, alpha: float = 0.7):
        self.model, self.beams, self.alpha = model, beams, alpha
        B, device = len(prompts), "cuda"
        self.ends = torch.tensor(ends, dtype=torch.int32, device=device)
        self.longest = max(len(p) for p in prompts)
        new = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=device)
        zeros = torch.zeros(B, dtype=torch.int32, device=device)
        table = torch.full((B, pages), -1, dtype=torch.int32, device=device)
        free = torch.arange(model.blocks, dtype=torch.int32, device=device)
        flat = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=device)
        logits, plan = model.step(flat, zeros, new, table, free, self.longest, 0)
        last = (plan.cu_new[1:] - 1).long()
        step = awq.beam_select(logits[last], torch.zeros((B, 1), device=device), beams, end_tokens=self.ends)
        self.history = torch.zeros((B * beams, 0), dtype=torch.int32, device=device)
        self.done_scores = torch.full((B, beams), -torch.inf, device=device)
        self.done_tokens = torch.full((B * beams, 0), -1, dtype=torch.int32, device=device)
        self.ones = torch.ones(B * beams, dtype=torch.int32, device=device)
        self._go_on(step, table, new, torch.zeros((B, 0), dtype=torch.int32, device=device), free, plan.counts[1:])

    def _go_on(self, step: awq.BeamStep, table, lens, history, free, start):
        B, W, parents = step.scores.shape[0], self.beams, step.parents.view(-1)
        # the candidates that ended here compete with those that ended before
        n = history.shape[1] + 1
        ended, = awq.reorder_states([history], step.ended_parents.view(-1))
        ended = torch.cat([ended, step.ended_tokens.view(-1, 1)], 1).view(B, W, n)
        before = torch.nn.functional.pad(self.done_tokens, (0, n - self.done_tokens.shape[1]), value=-1).view(B, W, n)
        scores, order = torch.cat([self.done_scores, step.ended_scores / n ** self.alpha], 1).topk(W, -1)
        self.done_scores = scores
        self.done_tokens = torch.cat([before, ended], 1).gather(1, order[..., None].expand(-1, -1, n)).reshape(B * W, n)
        self.scores = step.scores
        kept, = awq.reorder_states([history], parents)
        self.history = torch.cat([kept, step.tokens.view(-1, 1)], 1)
        self.table, self.lens, self.free = self.model.fork(table, lens, parents, free, start)

    def step(self):
        # a beam that is none has token -1 and score -inf; any token will do for it
        tokens = self.history[:, -1].clamp(min=0)
        logits, plan = self.model.step(tokens, self.lens, self.ones, self.table, self.free, 1, self.longest)
        self.longest += 1
        step = awq.beam_select(logits, self.scores, self.beams, end_tokens=self.ends)
        self._go_on(step, self.table, self.lens + 1, self.history, self.free, plan.counts[1:])


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--beams", type=int, default=4)
    a = ap.parse_args()
    gen = torch.Generator().manual_seed(5)
    prompts = [torch.randint(VOCAB, (5 + 9 * b,), generator=gen).tolist() for b in range(a.requests)]
    pages = -(-(9 * a.requests + 5 + a.steps + 1) // PAGE)
    # while a step runs its beams have a block each beside those of the step before
    search = BeamSearch(Decoder(a.requests * (a.beams + 1) * (pages + 1)), prompts, a.beams, ends=[0, 1, 2], pages=pages)
    for _ in range(a.steps):
        search.step()
    for b in range(a.requests):
        best = search.history.view(a.requests, a.beams, -1)[b, 0].tolist()
        print(f"request {b}: score {search.scores[b, 0].item():.3f}, tokens {best}; "
              f"{int((search.done_scores[b] > -torch.inf).sum())} ended")
    status = awq.awq_last_device_status(torch.cuda.current_stream().cuda_stream)
    assert status == awq.Status.OK, awq.awq_status_string(status)


if __name__ == "__main__":
    main()
