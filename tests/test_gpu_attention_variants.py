"""Every kernel and row variant behind tg_attend_step on the paths that the small
cases reach in one of them only: bad pages, odd numbers of key heads, peaked
scores, equal bits, another stream, and a graph (in whose capture an
allocation would be an error)."""
import numpy as np
import pytest

from oracle import attention_oracle as A
from tests.attention_util import Cache, check_attention, f64, ids, step_reference, torch_types
from tests.test_gpu_attention_step import run_case

pytestmark = pytest.mark.gpu

# heads per key head, n, type, cache, page, layout
VARIANTS = [
    (4, 1, "bf16", "bf16", 16, "token"),    # up to 8 rows
    (4, 4, "f16", "f16", 32, "head"),       # 16 rows
    (4, 17, "bf16", "bf16", 16, "token"),   # tensor memory, one row tile
    (5, 32, "f16", "f16", 128, "head"),     # two row tiles
    (4, 1, "bf16", "e4m3", 16, "token"),
    (3, 4, "f16", "e4m3", 64, "head"),
    (4, 7, "bf16", "e4m3", 16, "token"),
    (4, 12, "f16", "e4m3", 32, "token"),
    (4, 17, "bf16", "e4m3", 16, "head"),
    (4, 1, "f16", "f16", 4, "token"),       # pages copied row by row
    (4, 17, "bf16", "bf16", 2, "head"),
]
NAMES = ["-".join(map(str, v)) for v in VARIANTS]


def setup(variant, lens, G=3, D=128, seed=20):
    import torch
    import logits_processing_token_gb300 as tg
    rep, n, typ, kind, page, layout = variant
    c = Cache(lens, G, D, kind, page, layout, seed)
    rng = np.random.default_rng(seed)
    scales = rng.uniform(0.02, 0.08, (2, G)).astype(np.float32) if kind == "e4m3" else (None, None)
    cfg = tg.AttnConfig(num_heads=G * rep, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype=kind, page_size=page,
                        page_layout=layout, k_scales=scales[0], v_scales=scales[1], max_step_tokens=32)
    q = torch.from_numpy(rng.normal(0, 2, (len(lens), n, G * rep, D)).astype(np.float32)).cuda().to(torch_types()[typ])
    return cfg, c, q, scales, torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")


@pytest.mark.parametrize("variant", VARIANTS, ids=NAMES)
def test_keys_of_bad_pages_are_left_out(variant):
    import torch
    import logits_processing_token_gb300 as tg
    rep, n, typ, kind, page, _ = variant
    lens = [700, 300, 130, 90]
    cfg, c, q, scales, out, lse = setup(variant, lens)
    keep = [np.ones(length, bool) for length in lens]
    table = c.device_table()
    total = c.k.shape[0]
    for b, key, bad in ((0, 10, -7), (0, 333, total), (0, 699, 10 ** 9), (1, 0, -1), (1, 150, total + 1), (2, 129, -2)):
        table[b, key // page] = bad
        keep[b][key // page * page:(key // page + 1) * page] = False
    kl = ids([700, 300, 130, table.shape[1] * page + 1], np.int32)  # the last: longer than its row of the table
    tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, out, lse)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_PAGE | tg.TG_FLAG_BAD_ROW
    assert (out[3] == 0).all() and torch.isneginf(lse[3]).all()
    qf, H = f64(q), q.shape[2]
    for b in range(3):
        for j in range(n):
            sees = np.flatnonzero(keep[b][:max(0, lens[b] - n + j + 1)])
            for g in range(H // rep):
                k, v = c.keys[b][sees, g], c.values[b][sees, g]
                if kind == "e4m3":
                    k, v = k * np.float64(scales[0][g]), v * np.float64(scales[1][g])
                heads = slice(g * rep, (g + 1) * rep)
                want = A.attend(qf[b, j, heads], k, v, [len(sees)] * rep, 1 / np.sqrt(128), typ, "f16" if kind == "e4m3" else typ)
                check_attention((out[b, j, heads], lse[b, j, heads]), want)


@pytest.mark.parametrize("case", [
    # heads, key heads, dim, type, cache, page, layout, n, lengths
    (12, 3, 128, "bf16", "bf16", 16, "token", 17, [2000, 5, 700, 0]),
    (15, 5, 64, "f16", "f16", 32, "head", 17, [1500, 40, 300]),
    (10, 5, 80, "bf16", "bf16", 8, "token", 32, [600, 31]),
    (3, 3, 96, "f16", "f16", 16, "token", 32, [900, 33]),
    (12, 3, 128, "bf16", "e4m3", 16, "head", 17, [900, 17]),
    (7, 7, 64, "bf16", "e4m3", 32, "token", 1, [1200, 0, 3]),
], ids=lambda c: "-".join(map(str, c[:8])))
def test_odd_numbers_of_key_heads(case):
    run_case(*case, seed=30)


def test_peaked_scores_of_many_rows():
    run_case(8, 2, 128, "bf16", "bf16", 16, "token", 17, [1500, 70], seed=31, grow=20.0)
    run_case(6, 3, 64, "f16", "f16", 16, "head", 20, [900, 70], seed=32, grow=20.0)
    run_case(8, 2, 128, "bf16", "e4m3", 16, "token", 17, [700, 70], seed=33, grow=20.0)


@pytest.mark.parametrize("variant", VARIANTS, ids=NAMES)
def test_equal_bits_on_a_stream_and_in_a_graph(variant):
    import torch
    import logits_processing_token_gb300 as tg
    lens = [2000, 0, 17, 900, 64]
    cfg, c, q, scales, out, lse = setup(variant, lens)
    kl, table = ids(lens, np.int32), c.device_table()
    call = lambda o, z: tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, o, z)  # noqa: E731
    call(out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, z2 = torch.empty_like(out), torch.empty_like(lse)
    with torch.cuda.stream(side):
        call(o2, z2)
    side.synchronize()
    assert torch.equal(o2, out) and torch.equal(z2, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(o2, z2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(z2, lse)
    now = np.array([33, 0, 0, 899, 1])
    kl.copy_(ids(now, np.int32))
    g.replay()
    torch.cuda.synchronize()
    rep, n, typ, kind = variant[:4]
    want = step_reference(c, f64(q), n, rep, 1 / np.sqrt(128), typ, "f16" if kind == "e4m3" else typ, *scales, lens=now)
    check_attention((o2, z2), want)
    assert tg.tg_attn_status_word(cfg) == 0
