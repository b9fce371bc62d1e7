"""The beam-search example, the step's operators and the quantised layers together: every beam's score is
the sum of the log-probabilities that the model gives its tokens when they are read in one piece, and
beams that share pages say what beams with caches of their own say.

Tolerance of a score: the two runs differ in the shapes of their matrix products, so each token's logits by
0.04 (1 + |logit|) at most (twenty fp16 roundings of values of order one, amplified by about four, as derived for
the example of drafted trees), its log-probability by twice that; a score sums `steps` of them.
"""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def search(ex, prompts, beams, steps, ends, seed=0):
    pages = -(-(max(len(p) for p in prompts) + steps + 2) // ex.PAGE)
    s = ex.BeamSearch(ex.Decoder(len(prompts) * (beams + 1) * (pages + 1), seed), prompts, beams, ends=ends, pages=pages)
    for _ in range(steps):
        s.step()
    return s


def log_probability(ex, prompt, tokens):
    """Of `tokens` behind `prompt`, read in one piece; and the largest logit."""
    model = ex.Decoder(64)
    text = torch.tensor(prompt + tokens, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.full((1, 32), -1, dtype=torch.int32, device="cuda")
    logits, _ = model.step(text, zero, zero + len(text), table, torch.arange(64, dtype=torch.int32, device="cuda"), len(text), 0)
    x = logits[len(prompt) - 1:-1].double()
    return torch.log_softmax(x, -1).gather(1, torch.tensor(tokens, device="cuda")[:, None]).sum().item(), x.abs().max().item()


@pytest.mark.parametrize("beams,ends", [(4, [0, 1, 2]), (1, [5]), (7, list(range(0, 1024, 128)))])
def test_scores_are_the_tokens_log_probabilities(gpu, beams, ends):
    import beam_decode as ex
    gen = torch.Generator().manual_seed(beams)
    prompts = [torch.randint(ex.VOCAB, (n,), generator=gen).tolist() for n in (3, 16, 41)]
    steps = 20
    s = search(ex, prompts, beams, steps, ends)
    history = s.history.view(3, beams, -1).tolist()
    done = s.done_tokens.view(3, beams, -1).tolist()
    assert gpu.awq_last_device_status(torch.cuda.current_stream().cuda_stream) == 0
    for b in range(3):
        assert len({tuple(h) for h in history[b]}) == beams and s.scores[b].tolist() == sorted(s.scores[b].tolist(), reverse=True)
        for w in {0, beams - 1}:
            want, size = log_probability(ex, prompts[b], history[b][w])
            assert len(history[b][w]) == steps + 1 and not set(history[b][w]) & set(ends)
            assert abs(want - s.scores[b, w].item()) <= (steps + 1) * 2 * 0.04 * (1 + size)
        if s.done_scores[b, 0] > -torch.inf:
            tokens = [t for t in done[b][0] if t >= 0]
            want, size = log_probability(ex, prompts[b], tokens)
            assert tokens[-1] in ends and not set(tokens[:-1]) & set(ends)
            assert abs(want - s.done_scores[b, 0].item() * len(tokens) ** s.alpha) <= len(tokens) * 2 * 0.04 * (1 + size)


def test_one_beam_says_what_the_most_likely_tokens_say(gpu):
    import beam_decode as ex
    prompt = [7, 8, 9, 500]
    s = search(ex, [prompt], 1, 15, [1023])
    said = list(prompt)
    for t in s.history[0].tolist():
        model = ex.Decoder(64)
        text = torch.tensor(said, dtype=torch.int32, device="cuda")
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        table = torch.full((1, 32), -1, dtype=torch.int32, device="cuda")
        logits, _ = model.step(text, zero, zero + len(said), table, torch.arange(64, dtype=torch.int32, device="cuda"), len(said), 0)
        x = logits[-1].float()
        x[1023] = -torch.inf
        top = x.topk(2).values
        # only where the two best are closer than the tolerance may another be said
        assert t == x.argmax().item() or top[0] - x[t] <= 0.08 * (1 + top[0].abs())
        said.append(t)


def test_the_example_runs(gpu):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "beam_decode.py"), "--steps", "5"], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("request ") == 3
