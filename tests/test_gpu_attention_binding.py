"""The attention calls without the native marshalling module: the Python checks
pass them on, with the same bits."""
import numpy as np
import pytest

from tests.attention_util import ids

pytestmark = pytest.mark.gpu


def test_python_checks_alone_pass_the_calls_on():
    import torch
    import logits_processing_token_gb300 as tg
    H, G, D, P, n = 4, 2, 64, 16, [40, 7]
    g = torch.Generator("cuda").manual_seed(1)
    freq = (10000.0 ** (-np.arange(0, D, 2) / D)).tolist()
    qkv = torch.randn(sum(n), (H + 2 * G) * D, generator=g, device="cuda").bfloat16()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, G * D, G * D], dim=1))
    off, lens, table = ids([0, 40, 47], np.int64), ids(n, np.int32), ids([[4, 0, 2], [1, -1, -1]], np.int32)
    got = []
    for native in (True, False):
        cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, page_size=P, rotary_dim=D, inv_freq=freq)
        assert cfg._native is not None
        if not native:
            cfg._native = None
        kp, vp = (torch.zeros(5, P, G, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        qo, ko = torch.empty(47, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(47, G, D, dtype=torch.bfloat16, device="cuda")
        out, lse = torch.empty_like(qo), torch.empty(47, H, device="cuda")
        so, slse = torch.empty(2, 1, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, H, device="cuda")
        tg.tg_cache_append(q, k, v, off, lens, table, kp, vp, cfg, qo, ko)
        tg.tg_attend_prompt(qo, ko, v, off, None, cfg, out, lse)
        tg.tg_attend_step(qo[[39, 46]][:, None], lens, table, kp, vp, cfg, so, slse)
        torch.cuda.synchronize()
        got.append((kp, vp, qo, ko, out, lse, so, slse))
    for a, b in zip(*got):
        assert torch.equal(a, b)
