"""Speculative decoding with a small decoder of AWQ-quantised layers: a prompt
is filled in, then every step drafts a tree of tokens, checks all of its nodes in
one pass and keeps the longest path that the model itself would have taken.

The step's operators run as a serving process uses them: ``paged_plan`` lays the
step out from the request lengths, each layer appends its keys and values
(``kv_append``) and attends over the paged cache (``tree_attention``) between its
quantised projections, and ``process_logits`` applies penalties, biases and a
token mask to every node's logits.

    python examples/tree_decode.py [--steps 8] [--requests 3]
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


def rotate(x: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
    """Rotary position embedding of [tokens, heads, DIM]."""
    half = DIM // 2
    angle = positions[:, None].float() * 10000.0 ** (-torch.arange(half, device=x.device) / half)
    cos, sin = angle.cos()[:, None].to(x.dtype), angle.sin()[:, None].to(x.dtype)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).contiguous()


def norm(x: torch.Tensor) -> torch.Tensor:
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).half()


class Decoder:
    """Weights, the requests' paged caches and their lengths."""

    def __init__(self, requests: int, max_tokens: int, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)
        self.embedding = torch.randn((VOCAB, HIDDEN), generator=gen).half().cuda()
        self.layers = [(quantised_layer(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM, seed + 4 * i),
                        quantised_layer(HIDDEN, HIDDEN, seed + 4 * i + 1)) for i in range(LAYERS)]
        self.head = quantised_layer(HIDDEN, VOCAB, seed + 99)
        pages = -(-max_tokens // PAGE)
        self.caches = [[torch.zeros((requests * pages, PAGE, KV_HEADS, DIM), dtype=torch.float16, device="cuda")
                        for _ in range(2)] for _ in range(LAYERS)]
        self.table = torch.full((requests, pages), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(requests * pages, generator=gen).to(torch.int32).cuda()
        self.lengths = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.longest = 0                   # a bound of the lengths, known without asking the GPU

    def step(self, tokens: torch.Tensor, new: list[int], parents: torch.Tensor | None = None):
        """Logits [tokens, VOCAB] of the new tokens of all requests and the step's plan."""
        new_lens = torch.tensor(new, dtype=torch.int32).cuda()
        words = -(-max(new) // 32) if parents is not None else 0
        plan = awq.paged_plan(self.lengths, new_lens, self.table, self.free, PAGE, tokens.numel(), parents=parents,
                              mask_words=words)
        x = self.embedding[tokens.long()]
        for (qkv, out), (k_cache, v_cache) in zip(self.layers, self.caches):
            y = qkv(norm(x)).view(-1, HEADS + 2 * KV_HEADS, DIM)
            q = rotate(y[:, :HEADS], plan.positions)
            k = rotate(y[:, HEADS:HEADS + KV_HEADS], plan.positions)
            awq.kv_append(k, y[:, HEADS + KV_HEADS:], k_cache, v_cache, plan.slot_map)
            a = awq.tree_attention(q, k_cache, v_cache, self.table, self.lengths, plan.cu_new, DIM ** -0.5,
                                   max(new), self.longest, tree_mask=plan.tree_mask)
            x = x + out(a.view(-1, HIDDEN))
        return self.head(norm(x)), plan

    def keep(self, plan: awq.PagedPlan, paths: list[list[int]], new: list[int], drafted: bool):
        """Makes the tokens of `paths` (indices of new tokens, a path a request) the end of the
        requests: their keys and values move to the places right behind the context, and
        the pages that the step took and the requests no longer need become free again."""
        counts = plan.counts.tolist()
        if drafted:
            at = [sum(new[:b]) + i for b, path in enumerate(paths) for i in path]
            to = [sum(new[:b]) + j for b, path in enumerate(paths) for j in range(len(path))]
            for caches in self.caches:
                for cache in caches:
                    flat = cache.view(-1, KV_HEADS, DIM)
                    flat[plan.slot_map[to]] = flat[plan.slot_map[at]]
        self.free = self.free[counts[1]:]
        before = self.lengths.tolist()
        for b, path in enumerate(paths):
            kept, held = -(-(before[b] + len(path)) // PAGE), -(-(before[b] + new[b]) // PAGE)
            self.free = torch.cat([self.free, self.table[b, kept:held]])
        self.lengths += torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
        self.longest = max(n + len(p) for n, p in zip(before, paths))


class Sampling:
    """The controls of every request, and their histories."""

    def __init__(self, prompts: list[list[int]], banned: list[int]):
        n = len(prompts)
        self.history = [list(p) for p in prompts]
        self.prompt_lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32).cuda()
        self.repetition = torch.full((n,), 1.1, device="cuda")
        self.frequency = torch.full((n,), 0.2, device="cuda")
        self.presence = torch.full((n,), 0.1, device="cuda")
        allowed = torch.ones(VOCAB, dtype=torch.bool)
        allowed[banned] = False
        weight = 1 << torch.arange(32)
        words = (allowed.view(-1, 32).long() * weight).sum(-1)
        self.mask = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)[None].cuda()

    def choose(self, logits, plan, rows, draft_tokens=None):
        """The most likely token of every row after penalties and mask; a drafted row's
        history includes the nodes above it and itself."""
        offsets, flat = [0], []
        for h in self.history:
            flat += h
            offsets.append(len(flat))
        done = awq.process_logits(
            logits, row_request=rows, history=torch.tensor(flat, dtype=torch.int32).cuda(),
            history_offsets=torch.tensor(offsets, dtype=torch.int32).cuda(), prompt_lens=self.prompt_lens,
            repetition=self.repetition, frequency=self.frequency, presence=self.presence, draft_tokens=draft_tokens,
            cu_new=None if draft_tokens is None else plan.cu_new,
            tree_mask=None if draft_tokens is None else plan.tree_mask, grammar_mask=self.mask,
            grammar_rows=torch.zeros(logits.shape[0], dtype=torch.int32, device="cuda"))
        return done, done.argmax(-1).tolist()


def fill_prompts(model: Decoder, prompts: list[list[int]], sampling: Sampling):
    """Runs the prompts; the first token each request says."""
    new = [len(p) for p in prompts]
    logits, plan = model.step(torch.tensor([t for p in prompts for t in p], dtype=torch.int32).cuda(), new)
    ends = torch.tensor([sum(new[:b + 1]) - 1 for b in range(len(new))]).cuda()
    model.keep(plan, [list(range(n)) for n in new], new, drafted=False)
    rows = torch.arange(len(new), dtype=torch.int32, device="cuda")
    return sampling.choose(logits[ends].contiguous(), plan, rows)[1]


def draft(history: list[int], said: int, gen: torch.Generator, answer: list[int] | None):
    """A tree below the token that is certain: two branches of guesses, tokens seen
    after it before, else at random. `answer` (a test's) puts the right tokens on the second."""
    tokens, parents = [said], [-1]
    for branch in range(2):
        up, last = 0, said
        for depth in range(3):
            seen = [b for a, b in zip(history, history[1:]) if a == last]
            guess = seen[-1 - branch] if len(seen) > branch else int(torch.randint(VOCAB, (1,), generator=gen))
            if branch == 1 and answer is not None and depth < len(answer):
                guess = answer[depth]
            tokens.append(guess)
            parents.append(up)
            up, last = len(tokens) - 1, guess
    return tokens, parents


def generate(model: Decoder, prompts: list[list[int]], steps: int, banned: list[int], answers=None):
    """Tokens said by every request after `steps` speculative steps, and the logits of
    the rows that were kept."""
    sampling = Sampling(prompts, banned)
    gen = torch.Generator().manual_seed(1)
    said = fill_prompts(model, prompts, sampling)
    out = [[t] for t in said]
    kept_logits = [[] for _ in prompts]
    for _ in range(steps):
        trees = [draft(h + o, o[-1], gen, None if answers is None else answers[b][len(o):])
                 for b, (h, o) in enumerate(zip(sampling.history, out))]
        new = [len(t) for t, _ in trees]
        tokens = torch.tensor([t for tree, _ in trees for t in tree], dtype=torch.int32).cuda()
        parents = torch.tensor([p for _, ps in trees for p in ps], dtype=torch.int32).cuda()
        logits, plan = model.step(tokens, new, parents)
        done, best = sampling.choose(logits, plan, plan.token_request, draft_tokens=tokens)
        paths = []
        for b, (tree, ps) in enumerate(trees):
            first, path = sum(new[:b]), [0]
            while True:                    # the child that the model chose, if it was drafted
                want = best[first + path[-1]]
                down = [i for i in range(len(tree)) if ps[i] == path[-1] and tree[i] == want]
                if not down:
                    break
                path.append(down[0])
            paths.append(path)
            kept_logits[b] += [done[first + i] for i in path]
            sampling.history[b] += [tree[i] for i in path]
            out[b] += [tree[i] for i in path[1:]] + [want]
        model.keep(plan, paths, new, drafted=True)
    return out, kept_logits


def generate_one_by_one(model: Decoder, prompts: list[list[int]], count: int, banned: list[int]):
    """The same without drafts: a token a step."""
    sampling = Sampling(prompts, banned)
    said = fill_prompts(model, prompts, sampling)
    out = [[t] for t in said]
    logits_of = [[] for _ in prompts]
    rows = torch.arange(len(prompts), dtype=torch.int32, device="cuda")
    for _ in range(count):
        for b, o in enumerate(out):
            sampling.history[b].append(o[-1])
        new = [1] * len(prompts)
        logits, plan = model.step(torch.tensor([o[-1] for o in out], dtype=torch.int32).cuda(), new)
        done, best = sampling.choose(logits, plan, rows)
        model.keep(plan, [[0]] * len(prompts), new, drafted=False)
        for b, t in enumerate(best):
            out[b].append(t)
            logits_of[b].append(done[b])
    return out, logits_of


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--requests", type=int, default=3)
    a = ap.parse_args()
    gen = torch.Generator().manual_seed(5)
    prompts = [torch.randint(VOCAB, (5 + 9 * b,), generator=gen).tolist() for b in range(a.requests)]
    model = Decoder(a.requests, 512)
    out, _ = generate(model, prompts, a.steps, banned=[0, 1])
    for b, tokens in enumerate(out):
        print(f"request {b}: {len(prompts[b])} prompt tokens, {len(tokens)} said in {a.steps} steps: {tokens}")
    status = awq.awq_last_device_status(torch.cuda.current_stream().cuda_stream)
    assert status == awq.Status.OK, awq.awq_status_string(status)


if __name__ == "__main__":
    main()
