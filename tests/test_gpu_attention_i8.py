"""The i8 cache: tg_cache_append computes scales and codes as the definition says,
bit for bit; tg_attend_step over it against the 64-bit oracle."""
import numpy as np
import pytest

from oracle import attention_oracle as A
from tests.attention_util import check_attention, f64, ids, torch_types
from tests.quant_util import I8Cache, i8_reference, page_bytes, parts, quantised

pytestmark = pytest.mark.gpu


def append(H, G, D, typ, page, layout, new, lens, rotary=0, inter=False, extra=0, seed=0, grow=None, with_q=True, wide=0):
    """Append random tokens to an untouched cache; returns everything a check needs."""
    import torch
    import logits_processing_token_gb300 as tg
    c = I8Cache(lens, G, D, page, layout, seed, fill=False, extra=extra)
    rng = np.random.default_rng(seed + 1)
    T, t = int(sum(new)), torch_types()[typ]
    row = (H + 2 * G) * D + wide
    x = rng.normal(0, 1, (T, row)).astype(np.float32)
    if grow is not None:
        x[:, :(H + 2 * G) * D] = grow(x[:, :(H + 2 * G) * D].reshape(T, -1, D)).reshape(T, -1)
    qkv = torch.from_numpy(x).cuda().to(t)
    q, k, v = (y.unflatten(1, (-1, D)) for y in qkv[:, :(H + 2 * G) * D].split([H * D, G * D, G * D], dim=1))
    f = (10000.0 ** (-np.arange(0, rotary, 2) / max(rotary, 1))).astype(np.float32)
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype="i8", page_size=page, page_layout=layout,
                        rotary_dim=rotary, rotary_interleaved=inter, inv_freq=f.tolist() if rotary else None)
    off = ids(np.concatenate([[0], np.cumsum(new)]), np.int64)
    q_out, k_out = torch.empty(T, H, D, dtype=t, device="cuda"), torch.empty(T, G, D, dtype=t, device="cuda")
    before = [p.clone() for p in (c.k, c.v)]
    tg.tg_cache_append(q if with_q else None, k, v, off, ids(lens, np.int32), c.device_table(), c.k, c.v, cfg,
                       q_out if with_q else None, k_out)
    torch.cuda.synchronize()
    pos = np.concatenate([np.arange(n - m, n) for m, n in zip(new, lens)]).astype(np.int64)
    seq = np.repeat(np.arange(len(new)), new)
    return dict(tg=tg, cfg=cfg, c=c, q=q, k=k, v=v, q_out=q_out, k_out=k_out, before=before, pos=pos, seq=seq, f=f, inter=inter,
                page=c.table[seq, pos // page], slot=pos % page, off=off)


def places(r, pool, G, D, page, layout):
    """(bytes [T, G, D], scales [T, G]) of the appended tokens."""
    codes, scales = (x.cpu().numpy() for x in parts(pool, G, D, page, layout))
    at = codes[r["page"], r["slot"]] if layout == "token" else codes[r["page"], :, r["slot"]]
    return at, scales[r["page"], :, r["slot"]]


def untouched(r, pool, before, G, D, page, layout):
    """Every byte that is no appended token's is as it was."""
    for p in (pool, before):
        codes, scales = parts(p, G, D, page, layout)
        pg, sl = ids(r["page"], np.int64), ids(r["slot"], np.int64)
        if layout == "token":
            codes[pg, sl] = 0
        else:
            codes[pg, :, sl] = 0
        scales[pg, :, sl] = 0.0
    return bool((pool == before).all())


EXACT = [
    # heads, key heads, dim, type, page, layout, new, lengths
    (4, 1, 128, "bf16", 16, "token", [1], [1]),
    (8, 2, 128, "f16", 16, "head", [3, 0, 40], [3, 5, 77]),
    (3, 3, 80, "bf16", 1, "token", [5, 1], [9, 1]),
    (5, 1, 96, "f16", 8, "head", [130], [200]),
    (2, 2, 16, "bf16", 2, "token", [7, 8], [7, 30]),
    (6, 2, 48, "f16", 4, "head", [1, 1, 1, 1], [1, 2, 64, 65]),
    (7, 7, 112, "bf16", 1024, "token", [700, 33], [1500, 40]),
    (40, 5, 64, "bf16", 32, "head", [9], [9]),
]


@pytest.mark.parametrize("case", EXACT, ids=lambda c: "-".join(map(str, c[:6])))
def test_append_bits(case):
    H, G, D, typ, page, layout, new, lens = case
    # rows of unlike size, some that lie on ties of the codes
    grow = lambda x: np.where(np.arange(x.shape[1])[None, :, None] % 2, np.round(x * 8) / 8, x * 37.0)  # noqa: E731
    r = append(H, G, D, typ, page, layout, new, lens, extra=32, grow=grow, wide=8)
    for x, pool, before in zip((r["k"], r["v"]), (r["c"].k, r["c"].v), r["before"]):
        got = places(r, pool, G, D, page, layout)
        want = quantised(x.float().cpu().numpy())
        assert np.array_equal(got[1].view(np.uint32), want[1].view(np.uint32))
        assert np.array_equal(got[0], want[0])
        assert untouched(r, pool, before, G, D, page, layout)
    import torch
    assert torch.equal(r["q_out"], r["q"]) and torch.equal(r["k_out"], r["k"])
    assert r["tg"].tg_attn_status_word(r["cfg"]) == 0


@pytest.mark.parametrize("H, G, D, typ, page, layout, rotary, inter", [
    (4, 2, 128, "bf16", 16, "token", 128, False), (4, 2, 128, "f16", 16, "head", 64, True), (6, 3, 80, "bf16", 8, "token", 40, False),
    (2, 1, 96, "f16", 64, "head", 24, False), (3, 1, 64, "bf16", 4, "token", 8, True)])
def test_append_rotated(H, G, D, typ, page, layout, rotary, inter):
    new, lens = [50, 1, 7], [50, 9000, 130000]
    if page < 8:
        lens = [50, 900, 1300]
    r = append(H, G, D, typ, page, layout, new, lens, rotary=rotary, inter=inter, seed=3)
    codes, scales = places(r, r["c"].k, G, D, page, layout)
    want, tol = A.rotate(f64(r["k"]), r["pos"], r["f"], inter)
    # the scale: the largest magnitude, off by its tolerance, over 127, one rounding
    top = np.abs(want).max(-1)
    assert (np.abs(scales - top / 127) <= tol.max(-1) / 127 + top / 127 * 2.0 ** -23).all()
    # the code: half a step of the scale and what the value, the scale and one rounding are off by
    value = (codes.astype(np.float64) - 128) * scales[..., None].astype(np.float64)
    assert (np.abs(value - want) <= scales[..., None] * (0.5 + 2.0 ** -15) + tol).all()
    q, qt = A.rotate(f64(r["q"]), r["pos"], r["f"], inter)
    assert (np.abs(f64(r["q_out"]) - q) <= A.rounded_tol(q, qt, typ)).all()
    v = places(r, r["c"].v, G, D, page, layout)
    exact = quantised(r["v"].float().cpu().numpy())
    assert np.array_equal(v[0], exact[0]) and np.array_equal(v[1], exact[1])


def test_append_extremes():
    # heads of zeros, of the smallest and largest numbers, with an infinity or a NaN: none spoils another
    import torch
    T, G, D = 12, 3, 64
    rows = np.random.default_rng(4).normal(0, 1, (T, 3 * G, D)).astype(np.float32)
    rows[0] = 0.0
    rows[1] *= 1e-39
    rows[2] = np.float32(2.0 ** -133)
    rows[3] *= 5e37
    rows[4, :, 5] = np.inf
    rows[5, :, 6] = -np.inf
    rows[6, :, 7] = np.nan
    rows[7, :, 1:] = 0.0
    rows[8, :, 0] = 3e38
    rows[9, :, 0] = -0.0
    rows[10] *= np.where(np.arange(D) % 2, 1.0, 1e-30)
    r = append(G, G, D, "bf16", 16, "token", [T], [T], seed=4, grow=lambda x: rows)
    for x, pool in zip((r["k"], r["v"]), (r["c"].k, r["c"].v)):
        codes, scales = places(r, pool, G, D, 16, "token")
        q, s = quantised(x.float().cpu().numpy())
        assert np.isnan(scales[4:7]).all() and (codes[4:7] == 128).all()
        keep = [t for t in range(T) if t not in (4, 5, 6)]
        assert np.array_equal(scales[keep], s[keep]) and np.array_equal(codes[keep], q[keep])
        assert (scales[0] == 0).all() and (codes[0] == 128).all()
    k = torch.empty_like(r["k_out"])
    r["tg"].tg_cache_read(r["off"], ids([T], np.int32), r["c"].device_table(), r["c"].k, r["c"].v, r["cfg"], k)
    assert torch.isnan(k[4:7]).all() and torch.isfinite(k[[0, 1, 2, 3, 7, 8, 9, 10, 11]]).all()


def test_append_keeps_to_its_rows():
    # no query; a page outside the cache, a length shorter than the new tokens: flagged, skipped, the rest written
    import torch
    import logits_processing_token_gb300 as tg
    H, G, D, P = 2, 2, 64, 16
    c = I8Cache([40, 30, 5], G, D, P, "token", 7, fill=False)
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, cache_dtype="i8", page_size=P)
    kv = torch.randn(2, 75, G, D, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    table = c.device_table()
    table[0, 1] = 10 ** 6
    lens = ids([40, 30, 3], np.int32)  # two of the last sequence's five tokens have no position
    k0, v0 = c.k.clone(), c.v.clone()
    tg.tg_cache_append(None, kv[0], kv[1], ids([0, 40, 70, 75], np.int64), lens, table, c.k, c.v, cfg)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_PAGE | tg.TG_FLAG_BAD_ROW
    seq = np.repeat([0, 1, 2], [40, 30, 5])
    pos = np.concatenate([np.arange(40), np.arange(30), np.arange(-2, 3)])
    good = (pos >= 0) & ~((seq == 0) & (pos // P == 1))
    r = dict(page=c.table[seq[good], pos[good] // P], slot=pos[good] % P)
    for x, pool, before in ((kv[0], c.k, k0), (kv[1], c.v, v0)):
        want = quantised(x.float().cpu().numpy()[good])
        got = places(r, pool, G, D, P, "token")
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert untouched(r, pool, before, G, D, P, "token")


STEP = [
    # heads, key heads, dim, type, page, layout, n, lengths
    (4, 1, 128, "bf16", 16, "token", 1, [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 300]),
    (8, 2, 128, "bf16", 64, "head", 1, [1000, 3, 0, 129]),
    (16, 2, 64, "f16", 32, "head", 1, [5, 700, 64]),
    (3, 3, 64, "f16", 8, "token", 1, [1, 33, 511]),
    (32, 2, 128, "bf16", 64, "head", 1, [300, 0, 1, 77]),
    (5, 1, 80, "bf16", 16, "token", 1, [40, 300]),
    (6, 2, 96, "f16", 1, "token", 1, [70, 9]),
    (4, 2, 80, "bf16", 1024, "head", 1, [100, 1500]),
    (2, 2, 16, "bf16", 2, "head", 1, [65, 4]),
    (7, 1, 112, "f16", 4, "token", 2, [1, 2, 3, 260]),
    (8, 2, 128, "bf16", 16, "token", 5, [0, 1, 4, 5, 6, 64, 67, 333]),
    (8, 2, 128, "bf16", 16, "token", 17, [16, 17, 18, 300, 2]),
    (32, 4, 128, "f16", 128, "head", 17, [20, 200]),
    (8, 1, 64, "f16", 32, "token", 9, [8, 9, 190]),
    (16, 1, 128, "bf16", 32, "token", 32, [31, 100]),
    (4, 4, 48, "bf16", 2, "head", 32, [40, 130]),
    (5, 5, 128, "f16", 16, "token", 23, [140, 0, 22, 23, 24]),
    (128, 1, 64, "bf16", 8, "token", 2, [9, 200]),
]


def run_step(H, G, D, typ, page, layout, n, lens, seed=0, spread=1.0, extra=0, grow=1.0, with_lse=True):
    import torch
    import logits_processing_token_gb300 as tg
    c = I8Cache(lens, G, D, page, layout, seed, extra=extra, spread=spread)
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype="i8", page_size=page, page_layout=layout,
                        max_step_tokens=32)
    t = torch_types()[typ]
    q = torch.from_numpy(np.random.default_rng(seed + 1).normal(0, 2 * grow, (len(lens), n, H, D)).astype(np.float32)).cuda().to(t)
    out = torch.full((len(lens), n, H, D), float("nan"), device="cuda", dtype=t)
    lse = torch.full((len(lens), n, H), float("nan"), device="cuda") if with_lse else None
    tg.tg_attend_step(q, ids(lens, np.int32), c.device_table(extra=3), c.k, c.v, cfg, out, lse)
    torch.cuda.synchronize()
    check_attention((out, lse), i8_reference(c, f64(q), n, H // G, 1 / np.sqrt(D), typ))
    assert tg.tg_attn_status_word(cfg) == 0
    return tg, cfg, c, q, out, lse


@pytest.mark.parametrize("case", STEP, ids=lambda c: "-".join(map(str, c[:7])))
def test_step_matches_oracle(case):
    run_step(*case, extra=48)


def test_step_long_and_many():
    run_step(4, 1, 128, "bf16", 64, "token", 1, [30_000], seed=5)
    run_step(2, 1, 64, "f16", 16, "token", 1, [int(x) for x in np.random.default_rng(6).integers(0, 40, 700)], seed=6)
    run_step(4, 1, 64, "f16", 16, "token", 20, [3000, 5], seed=7)
    run_step(6, 1, 128, "bf16", 16, "head", 22, [2500, 7, 0, 900], seed=8, with_lse=False)


@pytest.mark.parametrize("n", [1, 3, 17])
def test_step_scales_far_apart(n):
    # values whose scales differ by many orders, and peaked weights
    run_step(8, 2, 128, "bf16", 16, "token", n, [500, 70], seed=9, spread=6.0, grow=0.01)
    run_step(8, 2, 64, "f16", 16, "head", n, [500, 70], seed=10, spread=3.0, grow=0.2)
    run_step(8, 2, 128, "bf16", 16, "token", n, [400], seed=11, spread=0.0, grow=20.0)


def test_step_values_of_zeros_and_nan_keys():
    import torch
    tg, cfg, c, q, out, lse = run_step(4, 1, 64, "bf16", 16, "token", 1, [70, 100, 40], seed=12)
    codes, scales = parts(c.v, 1, 64, 16, "token")
    scales[ids(c.table[0, :5], np.int64)] = 0.0          # sequence 0: every value 0
    kscales = parts(c.k, 1, 64, 16, "token")[1]
    kscales[int(c.table[1, 2]), 0, 5] = float("nan")      # sequence 1 sees a key that is not a number
    tg.tg_attend_step(q, ids([70, 100, 40], np.int32), c.device_table(), c.k, c.v, cfg, out, lse)
    torch.cuda.synchronize()
    assert (out[0] == 0).all() and torch.isfinite(lse[0]).all()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    check_attention((out[2:], lse[2:]), [x[2:] for x in i8_reference(c, f64(q), 1, 4, 1 / 8, "bf16")])


@pytest.mark.parametrize("n, page", [(1, 16), (5, 16), (17, 16), (1, 4)])
def test_step_bad_pages(n, page):
    # keys of pages that do not exist are left out, whatever an earlier tile left behind
    import torch
    lens = [100, 40, 64, 500]
    tg, cfg, c, q, out, lse = run_step(8, 2, 64, "f16", page, "token", n, lens, seed=13)
    table = c.device_table()
    table[0, 32 // page] = 10 ** 6
    table[1, 0] = -5
    keep = [np.r_[0:32, 32 + page:100], np.r_[page:40], np.r_[0:64], np.r_[0:500]]
    tg.tg_attend_step(q, ids(lens, np.int32), table, c.k, c.v, cfg, out, lse)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_PAGE
    for x in (c.keys, c.values):
        for b in range(4):
            x[b] = x[b][keep[b]]
    check_attention((out, lse), i8_reference(c, f64(q), n, 4, 1 / 8, "f16", lens=np.array([len(k) for k in keep])))


def test_step_equal_bits_stream_and_graph():
    import torch
    lens = [2000, 0, 17, 900, 64]
    tg, cfg, c, q, out, lse = run_step(8, 2, 128, "bf16", 16, "token", 2, lens, seed=14)
    table, kl = c.device_table(), ids(lens, np.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, z2 = torch.empty_like(out), torch.empty_like(lse)
    tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, o2, z2, stream=side)
    side.synchronize()
    assert torch.equal(o2, out) and torch.equal(z2, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, o2, z2)
    for now in ([65, 30, 0, 1, 2], lens):
        now = [min(a, b) for a, b in zip(now, lens)]
        kl.copy_(ids(now, np.int32))
        g.replay()
        torch.cuda.synchronize()
        check_attention((o2, z2), i8_reference(c, f64(q), 2, 4, 1 / np.sqrt(128), "bf16", lens=np.array(now)))


def test_offsets_past_32_bits():
    # a pool of more than 2^31 bytes, the sequence at its far end: written, read back, attended
    import torch
    import logits_processing_token_gb300 as tg
    G, D, P, L = 8, 128, 64, 300
    size = page_bytes(P, G, D)
    pages = (1 << 31) // size + 40
    k, v = (torch.zeros(pages, size, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = ids(np.arange(pages - 1, pages - 1 - -(-L // P), -1)[None], np.int32)
    g = torch.Generator("cuda").manual_seed(1)
    q, kk, vv = (torch.randn(L, h, D, generator=g, device="cuda").bfloat16() for h in (8, G, G))
    cfg = tg.AttnConfig(num_heads=8, num_kv_heads=G, head_dim=D, page_size=P, cache_dtype="i8")
    off, kl = ids([0, L], np.int64), ids([L], np.int32)
    tg.tg_cache_append(None, kk, vv, off, kl, table, k, v, cfg)
    k2, v2 = torch.empty_like(kk), torch.empty_like(vv)
    tg.tg_cache_read(off, kl, table, k, v, cfg, k2, v2)
    c = I8Cache([0], G, D, P, "token", 0, fill=False)
    c.keys, c.values = [], []
    for x, y in ((kk, k2), (vv, v2)):
        codes, s = quantised(x.float().cpu().numpy())
        val = (codes.astype(np.float64) - 128) * s[..., None]
        assert (np.abs(f64(y) - val) <= np.abs(val) * (2.0 ** -8 + 2.0 ** -23)).all()
        (c.keys if x is kk else c.values).append(val)
    out, lse = torch.empty(1, 1, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, 8, device="cuda")
    last = q[-1][None, None].contiguous()
    tg.tg_attend_step(last, kl, table, k, v, cfg, out, lse)
    check_attention((out, lse), i8_reference(c, f64(last), 1, 1, 1 / np.sqrt(D), "bf16", lens=np.array([L])))


@pytest.mark.parametrize("rep, n, page", [(4, 1, 16), (4, 3, 16), (4, 17, 16), (4, 1, 4), (5, 32, 32)])
def test_step_after_waits_ran_out(rep, n, page):
    import torch
    import logits_processing_token_gb300 as tg
    from tests.test_gpu_attention_timeout import run_out
    lens, G, D = [3000, 40, 700, 0, 90], 3, 128
    c = I8Cache(lens, G, D, page, "token", 1)
    cfg = tg.AttnConfig(num_heads=G * rep, num_kv_heads=G, head_dim=D, cache_dtype="i8", page_size=page, max_step_tokens=32)
    q = torch.randn(len(lens), n, G * rep, D, generator=torch.Generator("cuda").manual_seed(2), device="cuda").bfloat16()
    kl, table, out = ids(lens, np.int32), c.device_table(), torch.empty_like(q)
    run_out(cfg, lambda: tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, out), out)
