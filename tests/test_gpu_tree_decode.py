"""The speculative-decoding example, the step's operators and the quantised layers
together: the logits of the tree's accepted nodes equal those of decoding one
token at a time, and so do the tokens.

Tolerance: the two runs differ in the shapes of their matrix products and in
their tilings, so every layer's fp16 outputs may differ in their last place and the
differences pass through two layers and the head: 2^-11 a rounding, about twenty
roundings of values of order one on the way, amplified by at most about four:
|a - b| <= 20 * 4 * 2^-11 (1 + |b|) = 0.04 (1 + |b|).
"""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_trees_say_what_one_by_one_decoding_says(gpu):
    import tree_decode as ex
    gen = torch.Generator().manual_seed(5)
    prompts = [torch.randint(ex.VOCAB, (n,), generator=gen).tolist() for n in (3, 17, 40)]
    want, want_logits = ex.generate_one_by_one(ex.Decoder(3, 256), prompts, 24, banned=[0, 7])
    # drafts that hold the right continuation on one branch: several tokens a step are kept
    got, got_logits = ex.generate(ex.Decoder(3, 256), prompts, 6, banned=[0, 7], answers=want)
    for b in range(3):
        n = min(len(got_logits[b]), len(want_logits[b]))
        assert n >= 12                       # drafts were accepted
        for i in range(n):
            x, y = got_logits[b][i].float(), want_logits[b][i].float()
            assert torch.equal(x == -torch.inf, y == -torch.inf)
            fine = y != -torch.inf
            assert ((x - y).abs() <= 0.04 * (1 + y.abs()))[fine].all()
            if got[b][i + 1] != want[b][i + 1]:
                # only where the two best were closer than the tolerance
                top = y.topk(2).values
                assert top[0] - top[1] <= 0.08 * (1 + top[0].abs())
                break
    assert gpu.awq_last_device_status(torch.cuda.current_stream().cuda_stream) == 0


def test_the_example_runs(gpu):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "tree_decode.py"), "--steps", "3"], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("request ") == 3
