"""examples/tree_decode.py: the cache, the attention and the verification together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decode.py")
    spec = importlib.util.spec_from_file_location("tree_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# Attention output and softmax weights are rounded to bfloat16 (2^-9 each, relative) in either of two
# layers; the logits have a scale of 4 and 256 or 512 products average the errors: 8 standard errors
# of 4 * 2 * 2^-9 * sqrt(2) are 0.18.
TOL = 0.18


@pytest.mark.parametrize("slots,prompt,page", [(1, 2, 8), (4, 150, 16), (5, 65, 64)])
def test_sequences_match_the_plain_model(slots, prompt, page):
    ex = _example()
    seqs, emitted, worst = ex.run(slots, 12, prompt, page)
    assert worst < TOL
    assert 1.0 <= emitted <= 5.0
    for s in seqs:
        assert len(s) >= prompt + 12 and s[:prompt] == seqs[0][:prompt]
    for s in seqs[::2]:  # greedy slots continue alike
        n = min(len(s), len(seqs[0]))
        assert s[:n] == seqs[0][:n]


def test_greedy_slot_emits_the_plain_models_choice():
    """Every token is the plain model's likeliest, or within rounding of it."""
    ex = _example()
    model = ex.Model(seed=3)
    seqs, _, _ = ex.run(1, 10, 40, 16, seed=3, model=model)
    s = torch.tensor(seqs[0], dtype=torch.int32, device="cuda")
    z = model.plain(s[None])[0, 39:-1]
    chosen = z.gather(1, s[40:].long()[:, None])[:, 0]
    assert float((z.max(1).values - chosen).max()) < 2 * TOL
