"""The scoring example runs, and its log probabilities are those of its logits."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_prints_a_line_per_token(lib):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "score_tokens.py"), "--tokens", "9", "--vocab", "3001"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("likeliest") == 8 and "log probability of the sequence" in r.stdout


def test_example_scores_match_its_logits(lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        from score_tokens import Scorer
    finally:
        sys.path.pop(0)
    model = Scorer(256, 384, 2, 2000, seed=3)
    tokens = torch.randint(0, 2000, (20,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    logits = model.logits(tokens)
    assert bool(torch.isfinite(logits).all()) and float(logits.std()) > 0.1
    lp, ent, ids, tlp = model.score(tokens, top_k=4)
    ref = torch.log_softmax(logits[:-1].double(), dim=1)
    assert torch.allclose(lp.double(), ref.gather(1, tokens[1:, None])[:, 0], atol=2e-5, rtol=0)
    assert torch.allclose(ent.double(), -(ref.exp() * ref).sum(dim=1), atol=5e-5, rtol=0)
    assert torch.allclose(tlp.double(), ref.topk(4, dim=1).values, atol=2e-5, rtol=0)
    assert lib.get_last_error() == 0
