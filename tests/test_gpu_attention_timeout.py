"""Waits of the attention kernels that run out (their limit shortened through
tg_set_wait_limit): the launch ends and raises TG_FLAG_TIMEOUT, and once the
handle is cleared the next call gives its usual bits."""
import numpy as np
import pytest

from tests.attention_util import Cache, ids, torch_types

pytestmark = pytest.mark.gpu

LIMITS = [1, 300, 1500, 5000]


def run_out(cfg, call, out):
    import torch
    import logits_processing_token_gb300 as tg
    call()
    want = out.clone()
    for limit in LIMITS:
        out.fill_(float("nan"))
        tg.tg_set_wait_limit(limit)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            tg.tg_set_wait_limit(0)
        word = tg.tg_attn_status_word(cfg)
        assert word == tg.TG_FLAG_TIMEOUT or (limit > 1 and word == 0)
        tg.tg_attn_clear_status(cfg)
        call()
        torch.cuda.synchronize()
        assert tg.tg_attn_status_word(cfg) == 0 and torch.equal(out, want), limit


# rows of up to 8, 16, an 8-bit cache's row variants, pages copied row by row, tensor memory
@pytest.mark.parametrize("rep, n, typ, kind, page", [
    (4, 1, "bf16", "bf16", 16), (4, 3, "f16", "f16", 16), (4, 1, "bf16", "e4m3", 64), (4, 7, "bf16", "e4m3", 16),
    (4, 17, "f16", "e4m3", 16), (4, 1, "bf16", "bf16", 4), (4, 17, "bf16", "bf16", 16), (5, 32, "f16", "f16", 32)])
def test_step_after_waits_ran_out(rep, n, typ, kind, page):
    import torch
    import logits_processing_token_gb300 as tg
    lens, G, D = [3000, 40, 700, 0, 90], 3, 128
    c = Cache(lens, G, D, kind, page, "token", 1)
    cfg = tg.AttnConfig(num_heads=G * rep, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype=kind, page_size=page,
                        max_step_tokens=32)
    g = torch.Generator("cuda").manual_seed(2)
    q = torch.randn(len(lens), n, G * rep, D, generator=g, device="cuda").to(torch_types()[typ])
    kl, table, out = ids(lens, np.int32), c.device_table(), torch.empty_like(q)
    run_out(cfg, lambda: tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, out), out)


@pytest.mark.parametrize("H, G, D, typ", [(4, 1, 128, "bf16"), (3, 3, 64, "f16")])
def test_prompt_after_waits_ran_out(H, G, D, typ):
    import torch
    import logits_processing_token_gb300 as tg
    nq = [700, 41, 1, 333, 1500]
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ)
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v = (torch.randn(sum(nq), h, D, generator=g, device="cuda").to(torch_types()[typ]) for h in (H, G, G))
    off, out = ids(np.concatenate([[0], np.cumsum(nq)]), np.int64), torch.empty_like(q)
    run_out(cfg, lambda: tg.tg_attend_prompt(q, k, v, off, None, cfg, out), out)
