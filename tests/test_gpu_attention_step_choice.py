"""Steps of 17 to 32 rows over 8-bit heads of at most 64 are the step kernel's, whose results do not depend on the
size of the pages: the same keys on pages of 16 and of 4 tokens, which no other kernel takes, give equal bits."""
import numpy as np
import pytest

from tests.attention_util import Cache, ids, torch_types
from tests.quant_util import I8Cache, page_bytes, parts

pytestmark = pytest.mark.gpu


def quarters(c, pool, G, D):
    """A pool of pages of 16 tokens as one of pages of 4."""
    import torch
    if c.kind == "e4m3":
        return pool.unflatten(1, (4, 4)).flatten(0, 1)
    codes, scales = parts(pool, G, D, 16, "token")
    small = torch.zeros(pool.shape[0] * 4, page_bytes(4, G, D), dtype=torch.uint8, device="cuda")
    to_codes, to_scales = parts(small, G, D, 4, "token")
    to_codes.copy_(codes.unflatten(1, (4, 4)).flatten(0, 1))
    to_scales.copy_(scales.unflatten(2, (4, 4)).transpose(1, 2).flatten(0, 1))
    return small


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("H, G, D, typ, n", [(8, 2, 64, "bf16", 5), (8, 2, 64, "f16", 8), (3, 3, 32, "bf16", 17), (20, 1, 48, "f16", 1)])
def test_rows_of_small_heads(kind, H, G, D, typ, n):
    import torch
    import logits_processing_token_gb300 as tg
    lens = [700, n, 40, 3000, 129]
    c = I8Cache(lens, G, D, 16, "token", 81) if kind == "i8" else Cache(lens, G, D, kind, 16, "token", 81)
    q = torch.randn(len(lens), n, H, D, generator=torch.Generator("cuda").manual_seed(82), device="cuda").to(torch_types()[typ]) * 2
    got = []
    for page in (16, 4):
        cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype=kind, page_size=page, max_step_tokens=32)
        k, v, table = c.k, c.v, c.table
        if page == 4:
            k, v = quarters(c, k, G, D), quarters(c, v, G, D)
            table = (np.repeat(table, 4, 1) * 4 + np.arange(4 * table.shape[1]) % 4).clip(-1)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        tg.tg_attend_step(q, ids(lens, np.int32), ids(table, np.int32), k, v, cfg, out, lse)
        torch.cuda.synchronize()
        assert tg.tg_attn_status_word(cfg) == 0
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
