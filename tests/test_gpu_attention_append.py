"""tg_cache_append against the 64-bit oracle: rotation at near and far
positions, both pairings, every cache type and page order."""
import numpy as np
import pytest

from oracle import attention_oracle as A
from tests.attention_util import f64, ids, torch_types

pytestmark = pytest.mark.gpu

CASES = [
    # heads, key heads, dim, type, cache, page, layout, rotary, interleaved, new tokens, lengths
    (8, 2, 128, "bf16", "bf16", 16, "token", 128, False, [1, 1, 1], [1, 16, 4000]),
    (4, 4, 64, "f16", "f16", 8, "head", 64, True, [3, 0, 17, 1], [3, 5, 40, 1]),
    (4, 1, 128, "bf16", "e4m3", 64, "head", 64, False, [100, 1], [130, 7]),
    (6, 2, 80, "f16", "e4m3", 1, "token", 48, True, [9, 30], [9, 300]),
    (6, 2, 80, "f16", "f16", 32, "head", 40, False, [9, 30, 1], [9, 300, 70]),
    (4, 4, 80, "bf16", "e4m3", 16, "token", 40, True, [3, 20], [3, 25]),
    (3, 1, 16, "bf16", "e4m3", 16, "token", 8, False, [3, 20], [3, 25]),
    (2, 1, 96, "bf16", "bf16", 32, "token", 0, False, [5, 40], [50, 40]),
    (1, 1, 16, "f16", "f16", 2, "head", 16, False, [7], [9]),
    (40, 8, 128, "bf16", "bf16", 16, "token", 128, True, [700, 1, 2000], [700, 90, 5000]),
    (4, 2, 128, "f16", "f16", 1024, "token", 128, False, [2, 2], [1 << 24, 100_000_000]),
]


def run_case(H, G, D, typ, kind, page, layout, rotary, inter, new, lens, seed=0, with_q=True, with_k=True, inplace=False):
    import torch
    import logits_processing_token_gb300 as tg
    rng = np.random.default_rng(seed)
    t, ct = torch_types()[typ], torch_types()[kind]
    new, lens = np.array(new), np.array(lens)
    T, B = int(new.sum()), len(new)
    q8 = kind == "e4m3"
    ks = rng.uniform(0.01, 0.05, G).astype(np.float32) if q8 else None
    vs = rng.uniform(0.001, 0.05, G).astype(np.float32) if q8 else None  # the smallest saturate
    freq = (10000.0 ** (-np.arange(0, rotary, 2) / max(rotary, 1))).astype(np.float32)
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype=kind, page_size=page,
                        page_layout=layout, rotary_dim=rotary, rotary_interleaved=inter, inv_freq=freq, k_scales=ks,
                        v_scales=vs)
    qkv = torch.from_numpy(rng.normal(0, 1, (T, (H + 2 * G) * D + 8)).astype(np.float32)).cuda().to(t)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv[:, :-8].split([H * D, G * D, G * D], dim=1))
    if inplace:
        q = q.contiguous()
    first = (lens - new) // page
    count = int(((lens - 1) // page - first + 1).clip(0).sum()) + 2
    table = np.full((B, int((lens.max() - 1) // page) + 1), -1, np.int32)
    order, at = rng.permutation(count), 0
    for b in range(B):
        for i in range(first[b], -(-lens[b] // page)):
            table[b, i] = order[at]
            at += 1
    shape = (count, page, G, D) if layout == "token" else (count, G, page, D)
    kp = torch.randn(shape, device="cuda").to(ct)
    vp = torch.randn(shape, device="cuda").to(ct)
    before = f64(kp), f64(vp)
    qin = f64(q)
    qo = q if inplace else torch.full((T, H, D), float("nan"), device="cuda", dtype=t)
    ko = torch.full((T, G, D), float("nan"), device="cuda", dtype=t)
    off = np.concatenate([[0], np.cumsum(new)])
    args = (ids(off, np.int64), ids(lens, np.int32), ids(table, np.int32), kp, vp, cfg)
    tg.tg_cache_append(q if with_q else None, k, v, *args, q_out=qo if with_q else None, k_out=ko if with_k else None)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == 0
    pos = np.concatenate([np.arange(e - n, e) for n, e in zip(new, lens)]).astype(np.int64)
    seq = np.repeat(np.arange(B), new)
    kr, ktol = A.rotate(f64(k), pos, freq, inter)
    if with_q:
        qr, qtol = A.rotate(qin, pos, freq, inter)
        assert (np.abs(f64(qo) - qr) <= A.rounded_tol(qr, qtol, typ)).all()
    if with_k:
        assert (np.abs(f64(ko) - kr) <= A.rounded_tol(kr, ktol, typ)).all()
    page_of, slot = table[seq, pos // page], pos % page
    for pages, old, x, tol, sc in ((kp, before[0], kr, ktol, ks), (vp, before[1], f64(v), np.zeros_like(kr), vs)):
        got = f64(pages)
        if layout == "head":
            got, old = got.swapaxes(1, 2), old.swapaxes(1, 2)
        if q8:
            s = sc.astype(np.float64)[None, :, None]
            x, tol = x / s, tol / s + np.abs(x / s) * 2 ** -22
            x = np.clip(x, -448, 448)
        assert (np.abs(got[page_of, slot] - x) <= A.rounded_tol(x, tol, kind)).all()
        rest = np.ones(got.shape[:2], bool)
        rest[page_of, slot] = False
        assert np.array_equal(got[rest], old[rest], equal_nan=True)  # nothing else was written
    return cfg, (q, k, v), args, qo, ko


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:9])))
def test_append_matches_oracle(case):
    run_case(*case)


def test_append_without_outputs_and_in_place():
    run_case(4, 2, 64, "bf16", "bf16", 16, "token", 64, False, [5, 3], [5, 20], seed=1, with_q=False)
    run_case(4, 2, 64, "bf16", "bf16", 16, "token", 64, False, [5, 3], [5, 20], seed=2, with_k=False)
    run_case(4, 2, 64, "f16", "f16", 16, "token", 32, True, [5, 3], [5, 20], seed=3, inplace=True)


def test_append_flags_bad_pages_and_positions():
    import torch
    import logits_processing_token_gb300 as tg
    cfg, (q, k, v), args, qo, ko = run_case(4, 2, 64, "bf16", "bf16", 16, "token", 64, False, [5, 3, 2], [5, 20, 30], seed=4)
    off, lens, table, kp, vp, _ = args
    was = kp.clone(), vp.clone(), ko.clone()
    bad = table.clone()
    bad[0, 0] = kp.shape[0]
    bad[1, 1] = -1
    kp.zero_(), vp.zero_(), ko.zero_()
    tg.tg_cache_append(q, k, v, off, lens, bad, kp, vp, cfg, qo, ko)
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_PAGE
    tg.tg_attn_clear_status(cfg)
    assert torch.equal(ko, was[2])                     # rotated all the same
    assert int((kp != 0).any(-1).any(-1).sum()) == 2   # the tokens of sequence 2 alone
    # a length shorter than the new tokens: the first of them has no position, and the second one's, 0, lies in a
    # page that the table does not have
    short = lens.clone()
    short[2] = 1
    tg.tg_cache_append(q, k, v, off, short, table, kp, vp, cfg, qo, ko)
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_ROW | tg.TG_FLAG_BAD_PAGE
    tg.tg_attn_clear_status(cfg)
    # offsets that leave some tokens to no sequence
    odd = off.clone()
    odd[3] = 8
    tg.tg_cache_append(q, k, v, odd, lens, table, kp, vp, cfg, qo, ko)
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_ROW


def test_append_in_a_graph():
    import torch
    import logits_processing_token_gb300 as tg
    cfg, (q, k, v), args, qo, ko = run_case(4, 2, 64, "bf16", "e4m3", 16, "head", 64, False, [5, 3], [5, 20], seed=5)
    kp, want = args[3], args[3].clone().view(torch.uint8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tg.tg_cache_append(q, k, v, *args, q_out=qo, k_out=ko)
    q1 = qo.clone()
    qo.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, q1) and torch.equal(kp.view(torch.uint8), want)


def e4m3_case(scales, x):
    """x [T, G, D] (exact in bf16) as keys and values of a head-major e4m3 cache with these scales; both pools as f32."""
    import torch
    import logits_processing_token_gb300 as tg
    T, G, D = x.shape
    cfg = tg.AttnConfig(num_heads=G, num_kv_heads=G, head_dim=D, cache_dtype="e4m3", page_size=16, page_layout="head",
                        k_scales=scales, v_scales=scales)
    kv = x.cuda().bfloat16()
    assert torch.equal(kv.double().cpu().nan_to_num(), x.nan_to_num())
    pages = -(-T // 16)
    kp, vp = (torch.zeros(pages, G, 16, D, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    tg.tg_cache_append(None, kv, kv, ids([0, T], np.int64), ids([T], np.int32), ids(np.arange(pages)[None], np.int32), kp, vp, cfg)
    assert tg.tg_attn_status_word(cfg) == 0
    return [p.float().cpu().transpose(1, 2).reshape(-1, G, D)[:T] for p in (kp, vp)]


def test_append_e4m3_ties_go_to_even():
    # quotients halfway between two codes, with scales whose reciprocals are not exact
    import torch
    scales = [m / 64 for m in (3, 5, 6, 7)] + [0.1015625]  # 0.1015625 = 13 / 128
    odd = torch.arange(17, 32, 2).double()                # 5 bits: the middle of two codes of 4 bits
    t = torch.stack([torch.cat([odd, -odd]) * 2.0 ** e for e in range(-8, 3)])  # [T, 16]
    x = t[:, None] * torch.tensor(scales).double()[None, :, None]
    keep = x.bfloat16().double() == x                     # (13 times 5 bits can take 9)
    x = torch.where(keep, x, torch.zeros_like(x))
    want = torch.where(keep, t[:, None].expand_as(x), torch.zeros_like(x)).float().to(torch.float8_e4m3fn).float()
    for got in e4m3_case(scales, x):
        assert torch.equal(got, want)


def test_append_e4m3_scales_at_the_ends_of_f32():
    # a scale whose reciprocal is no f32 number, and one whose reciprocal is subnormal
    import torch
    tiny, huge = 2.0 ** -140, 3 * 2.0 ** 126
    row = torch.tensor([0.0, -0.0, 1.0, -1.0, 2.0 ** -133, 2.0 ** 125, 3.0 * 2.0 ** -132, 0.5] * 2).double()
    x = row[None, None].expand(3, 2, 16)
    want = (x / torch.tensor([tiny, huge]).double()[:, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn).float()
    for got in e4m3_case([tiny, huge], x):
        assert torch.equal(got, want)


def test_append_e4m3_is_the_rounded_quotient_of_every_value():
    # every bf16 number by many scales, against the division of f32 numbers, code by code
    import torch
    rng = np.random.default_rng(21)
    scales = np.concatenate([[448.0, 1.0, 1.9999999, 1.0000001, 2.0 ** -64, 2.0 ** 64, 3.4e38, 2.0 ** -149],
                             np.exp(rng.uniform(np.log(1e-3), np.log(10), 16)), 2.0 ** rng.uniform(-149, 127, 8)]).astype(np.float32)
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = every.double()[torch.isfinite(every)].view(-1, 1, 16).expand(-1, len(scales), 16)
    s = torch.from_numpy(scales)[:, None]
    want = (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for got in e4m3_case(scales.tolist(), x):
        assert torch.equal(got.to(torch.float8_e4m3fn).view(torch.uint8), want)


def test_append_e4m3_saturates_infinities_and_keeps_nan():
    import torch
    inf = float("inf")
    x = torch.tensor([inf, -inf, float("nan"), 1.0] * 4).double().view(1, 1, 16).expand(2, 3, 16)
    for got in e4m3_case([0.5, 2.0 ** -100, 2.0 ** 100], x):
        assert (got[..., 0::4] == 448).all() and (got[..., 1::4] == -448).all() and torch.isnan(got[..., 2::4]).all()
