"""tg_cache_read: what a cache holds, packed: every cache type and layout, some of the
tokens, strided outputs, bad pages and rows, streams and graphs."""
import numpy as np
import pytest

from tests.attention_util import Cache, f64, ids, torch_types
from tests.quant_util import I8Cache, parts

pytestmark = pytest.mark.gpu

CASES = [
    # key heads, dim, type, cache, page, layout, lengths, tokens of each that are read (None: all)
    (1, 128, "bf16", "bf16", 16, "token", [1], None),
    (8, 128, "bf16", "bf16", 16, "token", [100, 0, 33, 1000], None),
    (16, 64, "f16", "f16", 32, "head", [517], None),
    (3, 80, "bf16", "e4m3", 8, "head", [70, 9], [3, 9]),
    (2, 16, "f16", "e4m3", 1, "token", [5, 40], [0, 40]),
    (5, 96, "f16", "i8", 64, "head", [300, 1, 64, 65], None),
    (8, 128, "bf16", "i8", 16, "token", [2000, 31, 0], [7, 31, 0]),
    (1, 112, "bf16", "i8", 2, "head", [33], [20]),
    (7, 48, "f16", "f16", 1024, "token", [1500, 3], [1400, 1]),
]


def setup(G, D, typ, kind, page, layout, lens, seed=0):
    import logits_processing_token_gb300 as tg
    c = I8Cache(lens, G, D, page, layout, seed, extra=16) if kind == "i8" else Cache(lens, G, D, kind, page, layout, seed)
    rng = np.random.default_rng(seed + 1)
    ks, vs = (rng.uniform(0.02, 0.08, (2, G)) if kind == "e4m3" else (None, None))
    cfg = tg.AttnConfig(num_heads=G, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype=kind, page_size=page, page_layout=layout,
                        k_scales=ks, v_scales=vs)
    return tg, c, cfg, ks, vs


def wanted(c, which, scales, typ, kind, take):
    """What the tokens stand for: one f32 product, one rounding."""
    import torch
    rows = []
    for b, m in enumerate(take):
        x = (c.keys if which == 0 else c.values)[b]
        rows.append(x[len(x) - m:])
    x = torch.from_numpy(np.concatenate(rows))
    if kind == "e4m3":
        x = x * torch.from_numpy(np.asarray(scales, np.float32).astype(np.float64))[:, None]
    return x.float().to(torch_types()[typ])  # (code * scale: under 48 bits, exact in f64; one rounding to f32)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_read_bits(case):
    import torch
    G, D, typ, kind, page, layout, lens, take = case
    take = list(lens) if take is None else take
    tg, c, cfg, ks, vs = setup(G, D, typ, kind, page, layout, lens)
    T, t = sum(take), torch_types()[typ]
    off, kl, table = ids(np.concatenate([[0], np.cumsum(take)]), np.int64), ids(lens, np.int32), c.device_table(extra=2)
    k, v = torch.full((T, G, D), float("nan"), dtype=t, device="cuda"), torch.full((T, G, D), float("nan"), dtype=t, device="cuda")
    tg.tg_cache_read(off, kl, table, c.k, c.v, cfg, k, v)
    for which, x in enumerate((k, v)):
        assert torch.equal(x.cpu(), wanted(c, which, (ks, vs)[which], typ, kind, take))
    # keys and values side by side in wider rows, and each alone: what lies between is left alone
    both = torch.full((T, 2 * G * D + 16), 7.0, dtype=t, device="cuda")
    k2, v2 = both[:, :G * D].unflatten(1, (G, D)), both[:, G * D:2 * G * D].unflatten(1, (G, D))
    tg.tg_cache_read(off, kl, table, c.k, c.v, cfg, k2, None)
    assert torch.equal(k2, k) and (v2 == 7.0).all()
    k2.fill_(7.0)
    tg.tg_cache_read(off, kl, table, c.k, c.v, cfg, v=v2)
    assert torch.equal(v2, v) and (k2 == 7.0).all() and (both[:, 2 * G * D:] == 7.0).all()
    assert tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_read_bad_pages_and_rows(kind):
    import torch
    lens = [100, 40, 20]
    tg, c, cfg, ks, vs = setup(2, 64, "bf16", kind, 16, "token", lens, seed=2)
    table = c.device_table()
    table[0, 1] = 10 ** 6
    table[1, 2] = -1
    off = ids([0, 100, 140, 165], np.int64)  # five more than the last sequence has
    k, v = (torch.full((170, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tg.tg_cache_read(off, ids(lens, np.int32), table, c.k, c.v, cfg, k, v)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_PAGE | tg.TG_FLAG_BAD_ROW
    for which, x in enumerate((k, v)):
        want = wanted(c, which, (ks, vs)[which], "bf16", kind, lens)
        want[16:32] = 0
        want[100 + 32:140] = 0
        assert torch.equal(x[:140].cpu(), want[:140])
        assert (x[140:145] == 7.0).all() and torch.equal(x[145:165].cpu(), want[140:160]) and (x[165:] == 7.0).all()
    tg.tg_attn_clear_status(cfg)
    # offsets that run backwards and past the rows stay inside
    k.fill_(7.0)
    tg.tg_cache_read(ids([5, 3, 90, 10 ** 9], np.int64), ids(lens, np.int32), c.device_table(), c.k, c.v, cfg, k)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) & tg.TG_FLAG_BAD_ROW


def test_read_nan_and_infinity():
    # a 16-bit cache's bits as they are; an e4m3 NaN stays one; a scale of NaN is the row's alone
    import torch
    tg, c, cfg, _, _ = setup(1, 64, "bf16", "bf16", 16, "token", [20])
    c.k[int(c.table[0, 0]), 3, 0, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")], dtype=torch.bfloat16)
    k = torch.empty(20, 1, 64, dtype=torch.bfloat16, device="cuda")
    off, kl = ids([0, 20], np.int64), ids([20], np.int32)
    tg.tg_cache_read(off, kl, c.device_table(), c.k, c.v, cfg, k)
    assert k[3, 0, 0] == float("inf") and k[3, 0, 1] == float("-inf") and k[3, 0, 2].isnan() and torch.isfinite(k[:3]).all()
    tg, c, cfg, _, _ = setup(1, 64, "f16", "i8", 16, "token", [20])
    parts(c.k, 1, 64, 16, "token")[1][int(c.table[0, 0]), 0, 3] = float("nan")
    k = torch.empty(20, 1, 64, dtype=torch.float16, device="cuda")
    tg.tg_cache_read(off, kl, c.device_table(), c.k, c.v, cfg, k)
    assert k[3].isnan().all() and torch.isfinite(k[:3]).all() and torch.isfinite(k[4:]).all()


def test_read_stream_graph_and_append():
    # captured with the append in front of it: replays read what the replay wrote
    import torch
    G, D, lens = 4, 128, [60, 17]
    tg, c, cfg, _, _ = setup(G, D, "bf16", "i8", 16, "head", lens, seed=3)
    off, kl, table = ids([0, 5, 8], np.int64), ids(lens, np.int32), c.device_table()
    kv = torch.randn(2, 8, G, D, device="cuda").bfloat16()
    k, v = torch.empty_like(kv[0]), torch.empty_like(kv[1])

    def call():
        tg.tg_cache_append(None, kv[0], kv[1], off, kl, table, c.k, c.v, cfg)
        tg.tg_cache_read(off, kl, table, c.k, c.v, cfg, k, v)

    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        call()
    for seed in (1, 2):
        kv.copy_(torch.randn(kv.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(kv.float(), (k, v)):
            s = x.abs().amax(-1, keepdim=True) / 127
            # half a step of the scale and one rounding to bf16 (the product's own is below the 2^-7 that is left)
            assert ((y.float() - x).abs() <= s * 0.51 + x.abs() * 2.0 ** -8).all()
