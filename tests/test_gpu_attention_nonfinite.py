"""Infinities and NaN where a row of a step does not look, in every step kernel;
and NaN where it does."""
import numpy as np
import pytest

from tests.attention_util import Cache, ids, torch_types

pytestmark = pytest.mark.gpu

# heads per key head, n, type, cache, page: up to 8 rows, 16, the row variants of an 8-bit cache and of small pages, tensor memory
STEPS = [(4, 2, "bf16", "bf16", 16), (2, 5, "f16", "f16", 32), (4, 2, "bf16", "e4m3", 16), (2, 6, "bf16", "e4m3", 32),
         (4, 7, "f16", "e4m3", 16), (4, 12, "bf16", "e4m3", 64), (4, 17, "f16", "e4m3", 16), (2, 3, "bf16", "bf16", 4),
         (4, 17, "bf16", "bf16", 2), (4, 17, "bf16", "bf16", 16), (3, 20, "f16", "f16", 64), (5, 32, "bf16", "bf16", 32)]


def step(rep, n, typ, kind, page, lens, change, G=3, D=64):
    """One step over a cache whose keys and values `change` has gone over; (out, lse)."""
    import torch
    import logits_processing_token_gb300 as tg
    c = Cache(lens, G, D, kind, page, "token", 5)
    cfg = tg.AttnConfig(num_heads=G * rep, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype=kind, page_size=page,
                        max_step_tokens=32)
    q = torch.randn(len(lens), n, G * rep, D, generator=torch.Generator("cuda").manual_seed(6), device="cuda").to(torch_types()[typ])
    change(c)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    tg.tg_attend_step(q, ids(lens, np.int32), c.device_table(), c.k, c.v, cfg, out, lse)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == 0
    return out, lse


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_rows_without_keys_give_zero_whatever_the_values(case, bad):
    import torch
    n = case[1]
    lens = [1, n - 1, n, 3 * n]

    def values(c):
        c.v.copy_(torch.full(c.v.shape, bad, device="cuda").to(c.v.dtype))

    out, lse = step(*case, lens, values)
    for b, length in enumerate(lens):
        none = max(0, n - length)  # the first tokens see no key
        assert (out[b, :none] == 0).all() and torch.isneginf(lse[b, :none]).all()
        assert not torch.isfinite(out[b, none:].float()).any() or case[3] == "e4m3"  # inf saturates in an 8-bit cache
        assert torch.isfinite(lse[b, none:]).all()


def test_a_part_without_keys_does_not_touch_the_join():
    # 5 tiles of 128 keys twice over seven CTAs of two units each: the first sequence's last tile, of which its first
    # 15 tokens see nothing, is a part of its own
    import torch
    n, lens = 17, [514, 514]

    def values(c):
        c.v[ids(c.table[0][512 // 16:], np.int64)] = float("nan")

    out, lse = step(4, n, "bf16", "bf16", 16, lens, values, G=2)
    assert torch.isfinite(out[0, :15].float()).all() and torch.isfinite(lse[0]).all()
    assert torch.isnan(out[0, 15:]).all()


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_nan_keys_that_are_seen_give_nan(case):
    # of a short sequence, and of one whose parts several CTAs join
    import torch
    n = case[1]
    out, lse = step(*case, [n, 40, 3000], lambda c: c.k.copy_(torch.full(c.k.shape, float("nan"), device="cuda").to(c.k.dtype)))
    assert torch.isnan(out).all() and torch.isnan(lse).all()
