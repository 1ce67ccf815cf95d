"""examples/decode_step.py: the attention calls and token selection together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_verify_accepts_what_single_steps_decoded():
    ex = load()
    decoded, matches = ex.run(batch=3, new_tokens=6)
    assert decoded.shape == (3, 6) and (matches == 5).all()


def test_steps_agree_with_the_prompt_call():
    # the logits after a prompt, against those of its last token as a step over the same cache
    import torch
    ex = load()
    counts = torch.tensor([7, 40], device="cuda")
    ids = torch.randint(0, ex.VOCAB, (47,), device="cuda", dtype=torch.int32)
    whole = ex.Layer(2, 64, seed=3)
    want = whole.prompts(ids, counts)
    split = ex.Layer(2, 64, seed=3)
    keep = torch.ones(47, dtype=torch.bool, device="cuda")
    keep[[6, 46]] = False
    split.prompts(ids[keep], counts - 1)
    got = split.step(ids[[6, 46]][:, None])[:, 0]
    # attention rounded to bf16 on both sides, the weights by 2^-8 each: a few
    # units of bf16 in a sum of HEADS * DIM products of about unit variance
    assert (got - want).abs().max() <= 8 * 2.0 ** -8 * want.abs().max()
