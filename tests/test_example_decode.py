"""The decode-and-score example: the logprobs of the scored rollout are those of the distributions it was drawn from."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [dict(), dict(B=3, prompt=1, steps=5, V=4096, D=64), dict(B=1, prompt=700, steps=3, V=9001)])
def test_decode_and_score(sizes):
    spec = importlib.util.spec_from_file_location("decode_and_score", os.path.join(ROOT, "examples", "decode_and_score.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    out = example.run(**sizes)
    assert out["err"] == 0 and out["fault"] == 0
    assert (out["ids"] >= 0).all()                                # every token was drawn, none from behind a mask
    assert torch.isfinite(out["logp"]).all()
    # the decode's log-softmax is of fp32 logits, the score's of the same values in fp32: 2^-24 of |z| < 60 and of
    # |logp| < 60, and the forward's (16 M + 62) 2^-24 with M < 60
    assert (out["logp"] - out["drawn_logp"]).abs().max() < 2.0 ** -24 * (16 * 60 + 62 + 120)
    # each gradient row sums to g (1 - sum p) f / T up to the repeated tokens' factor; masked columns are 0
    assert torch.isfinite(out["dx"]).all() and out["dx"].abs().sum(1).min() > 0
