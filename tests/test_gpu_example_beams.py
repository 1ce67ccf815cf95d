"""examples/decode_step.py: chunks of a prompt and a beam search over a shared prompt, in a 16-bit and an i8 cache."""
import pytest

from tests.test_gpu_example import load

pytestmark = pytest.mark.gpu


def test_chunks_agree_with_the_whole_prompt():
    import torch
    ex = load()
    counts = torch.tensor([20, 40], device="cuda")
    ids = torch.randint(0, ex.VOCAB, (60,), generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.int32)
    want = ex.Layer(2, 64, seed=3).prompts(ids, counts)
    for kind, steps in ((None, 8), ("i8", 16)):
        layer = ex.Layer(2, 64, seed=3, cache_dtype=kind)
        layer.chunk(torch.cat([ids[:8], ids[20:35]]), torch.tensor([8, 15], device="cuda"))
        got = layer.chunk(torch.cat([ids[8:20], ids[35:]]), torch.tensor([12, 25], device="cuda"))
        # both sides in bf16, the weights by 2^-8 each, and half a step of 1 / 127 of the largest for an i8 key and
        # value (under 2^-7): a few units of bf16 in a sum of HEADS * DIM products of about unit variance
        assert (got - want).abs().max() <= steps * 2.0 ** -8 * want.abs().max()


@pytest.mark.parametrize("kind", [None, "i8"])
def test_beams_are_scored_as_their_tokens_are(kind):
    # each beam's score is the sum of its tokens' log-probabilities, from single steps over a cache of its own
    import torch
    ex = load()
    prompt = torch.randint(0, ex.VOCAB, (37,), generator=torch.Generator("cuda").manual_seed(2), device="cuda", dtype=torch.int32)
    tokens, scores = ex.beam_search(prompt, beams=4, new_tokens=5, seed=4, cache_dtype=kind)
    assert tokens.shape == (4, 5) and (scores[:-1] >= scores[1:]).all() and len({tuple(t) for t in tokens.tolist()}) == 4
    layer = ex.Layer(4, 64, seed=4, cache_dtype=kind)
    logits = layer.chunk(prompt.repeat(4), torch.full((4,), 37, device="cuda"))
    total = torch.zeros(4, device="cuda")
    for i in range(5):
        logp = torch.log_softmax(logits, -1)
        total += logp[torch.arange(4), tokens[:, i].long()]
        if i < 4:
            logits = layer.step(tokens[:, i:i + 1].contiguous())[:, 0]
    # five tokens, each off by what attention in bf16 (2^-8 of weights and output, on both sides) makes of the logits
    assert (total - scores).abs().max() <= 5 * 8 * 2.0 ** -8 * float(logits.abs().max())
