"""The status word of an attention handle, and its reset, next to calls in
flight on a stream that does not wait for the default one."""
import numpy as np
import pytest

from tests.attention_util import Cache, ids

pytestmark = pytest.mark.gpu


@pytest.fixture
def prompt():
    import torch
    import logits_processing_token_gb300 as tg
    g = torch.Generator("cuda").manual_seed(0)
    T, H, G, D = 6000, 16, 4, 128
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D)
    q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").bfloat16() for h in (H, G, G))
    off = torch.tensor([0, T], device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call(out, off=off):
        tg.tg_attend_prompt(q, k, v, off, None, cfg, out)
    return tg, torch, cfg, call, side, torch.empty_like(q)


def test_status_word_waits_for_calls_in_flight(prompt):
    tg, torch, cfg, call, side, out = prompt
    bad = torch.tensor([-1, 6000], device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):
            call(out)
        call(out, bad)
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_ROW
    tg.tg_attn_clear_status(cfg)
    assert tg.tg_attn_status_word(cfg) == 0


def test_clear_status_waits_for_prompts_in_flight(prompt):
    tg, torch, cfg, call, side, out = prompt
    call(out)
    torch.cuda.synchronize()
    o2, o3 = torch.full_like(out, float("nan")), torch.full_like(out, float("nan"))
    with torch.cuda.stream(side):
        for _ in range(4):
            call(o2)
    tg.tg_attn_clear_status(cfg)
    call(o3)
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(o3, out) and tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("n, rep", [(1, 4), (17, 4)])
def test_clear_status_waits_for_steps_in_flight(n, rep):
    import torch
    import logits_processing_token_gb300 as tg
    lens = [30_000, 41]
    c = Cache(lens, 2, 128, "bf16", 16, "token", 1)
    cfg = tg.AttnConfig(num_heads=2 * rep, num_kv_heads=2, head_dim=128)
    q = torch.randn(2, n, 2 * rep, 128, generator=torch.Generator("cuda").manual_seed(2), device="cuda").bfloat16()
    kl, table = ids(lens, np.int32), c.device_table()

    def call(out):
        tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, out)

    out = torch.empty_like(q)
    call(out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, o3 = torch.full_like(q, float("nan")), torch.full_like(q, float("nan"))
    with torch.cuda.stream(side):
        for _ in range(30):
            call(o2)
    tg.tg_attn_clear_status(cfg)
    call(o3)
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(o3, out) and tg.tg_attn_status_word(cfg) == 0
