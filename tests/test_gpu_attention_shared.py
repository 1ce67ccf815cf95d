"""tg_attend_shared against the 64-bit oracle: groups with a common prefix on shared pages
and on copies, rows that fill several tiles, short and empty sequences, groups of
one, offsets that are refused, pages that do not exist."""
import numpy as np
import pytest

from tests.attention_util import check_attention, f64, ids, step_reference, torch_types
from tests.quant_util import i8_reference, parts, shared_cache

pytestmark = pytest.mark.gpu

CASES = [
    # heads, key heads, dim, type, cache, page, layout, n, members, prefixes, own tokens of each sequence (0: an empty slot)
    (8, 2, 128, "bf16", "bf16", 16, "token", 1, [4], [200], [1, 5, 17, 40]),
    (8, 2, 128, "bf16", "bf16", 16, "token", 1, [2, 1, 3, 1], [130, 60, 16, 0], [1, 2, 3, 4, 200, 16, 15]),
    (6, 3, 64, "f16", "f16", 32, "head", 1, [5, 4], [1000, 33], [1, 0, 3, 64, 128, 1, 1, 1, 0]),
    (5, 1, 80, "bf16", "bf16", 8, "token", 1, [3, 2], [7, 8], [9, 1, 30, 2, 2]),
    (2, 2, 16, "f16", "f16", 16, "head", 1, [3], [300], [1, 1, 1]),
    (4, 1, 96, "f16", "f16", 64, "token", 1, [40], [129], [1 + i % 70 for i in range(40)]),
    (8, 2, 128, "bf16", "bf16", 16, "token", 5, [4, 3], [257, 128], [5, 6, 70, 5, 9, 5, 5]),
    (10, 2, 64, "bf16", "bf16", 16, "head", 9, [6], [150], [9, 10, 11, 12, 100, 9]),
    (20, 10, 80, "f16", "f16", 32, "head", 5, [3, 1, 2], [400, 10, 32], [5, 7, 60, 5, 5, 20]),
    (8, 2, 128, "bf16", "i8", 16, "token", 1, [4], [200], [1, 5, 17, 40]),
    (8, 1, 128, "f16", "i8", 64, "head", 1, [20, 3], [520, 64], [1 + 3 * i for i in range(23)]),
    (6, 3, 64, "bf16", "i8", 32, "token", 1, [5, 4], [1000, 33], [1, 0, 3, 64, 128, 1, 1, 1, 0]),
    (3, 3, 48, "f16", "i8", 8, "head", 2, [4, 2], [90, 17], [2, 3, 40, 2, 2, 9]),
    (8, 2, 128, "bf16", "i8", 128, "token", 6, [4, 3], [257, 128], [6, 7, 70, 6, 9, 6, 6]),
    (8, 2, 128, "bf16", "e4m3", 16, "token", 1, [4], [200], [1, 5, 17, 40]),
    (16, 2, 64, "f16", "e4m3", 32, "head", 1, [12, 2], [300, 40], [1 + i for i in range(14)]),
    (5, 5, 112, "bf16", "e4m3", 16, "head", 4, [4, 2], [100, 31], [4, 5, 6, 30, 4, 4]),
    (8, 1, 96, "f16", "e4m3", 64, "token", 3, [9], [333], [3 + 7 * i for i in range(9)]),
    (4, 2, 64, "bf16", "bf16", 4, "token", 1, [3], [50], [1, 2, 3]),          # pages too small to share
    (256, 1, 64, "bf16", "bf16", 16, "token", 1, [2], [60], [1, 2]),          # too many heads to share
    (128, 1, 64, "f16", "i8", 16, "head", 1, [3], [60], [1, 2, 9]),           # a token fills a tile
]


def room(c, heads, dim):
    """The page table with so many columns that the longest sequences it could name make sharing worth a launch."""
    import torch
    t = c.device_table()
    key = 2 * heads * dim  # bytes of an 8-bit key and value
    most = max(t.shape[1], -(-(120 << 20) // (key * c.page * t.shape[0])))
    wide = torch.full((t.shape[0], most), -1, dtype=torch.int32, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide


def setup(H, G, D, typ, kind, page, layout, n, members, prefix, own, seed=0, copies=False, lens=None, spare=0, small=False, **more):
    import torch
    import logits_processing_token_gb300 as tg
    own = np.asarray(own)
    pre = np.repeat(np.asarray(prefix), members)
    lens = np.where(own > 0, pre + own, 0) if lens is None else np.asarray(lens)
    c = shared_cache(kind, np.asarray(members), prefix, lens, G, D, page, layout, seed, copies=copies, **more)
    rng = np.random.default_rng(seed + 1)
    ks, vs = ((rng.uniform(0.02, 0.08, G).astype(np.float32)) for _ in range(2)) if kind == "e4m3" else (None, None)
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype=kind, page_size=page, page_layout=layout,
                        k_scales=ks, v_scales=vs, max_step_tokens=32, max_shared_tokens=len(lens) * n + spare)
    t = torch_types()[typ]
    q = torch.from_numpy(rng.normal(0, 2, (len(lens), n, H, D)).astype(np.float32)).cuda().to(t)
    off, pl = ids(np.concatenate([[0], np.cumsum(members)]), np.int64), ids(prefix, np.int32)
    c.table_now = lambda: c.device_table() if small else room(c, G, D)  # (small: too little to share)

    def reference(lens=None):
        if kind == "i8":
            return i8_reference(c, f64(q), n, H // G, 1 / np.sqrt(D), typ, lens=lens)
        return step_reference(c, f64(q), n, H // G, 1 / np.sqrt(D), typ, "f16" if kind == "e4m3" else typ, ks, vs, lens=lens)

    def call(out=None, lse=None, off=off, pl=pl, table=None, lens=lens, stream=None):
        out = torch.full((len(lens), n, H, D), float("nan"), device="cuda", dtype=t) if out is None else out
        lse = torch.full((len(lens), n, H), float("nan"), device="cuda") if lse is None else lse
        kl = lens if isinstance(lens, torch.Tensor) else ids(lens, np.int32)
        tg.tg_attend_shared(q, kl, c.table_now() if table is None else table, c.k, c.v, off, pl, cfg, out, lse, stream=stream)
        return out, lse

    return tg, cfg, c, q, off, pl, lens, reference, call


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:8])))
def test_shared_matches_oracle(case):
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(*case)
    out, lse = call()
    torch.cuda.synchronize()
    check_attention((out, lse), reference())
    assert tg.tg_attn_status_word(cfg) == 0
    o2, z2 = call()  # equal bits
    assert torch.equal(o2, out) and torch.equal(z2, lse)


@pytest.mark.parametrize("case", CASES[::3], ids=lambda c: "-".join(map(str, c[:8])))
def test_calls_too_small_to_share(case):
    tg, cfg, c, q, off, pl, lens, reference, call = setup(*case, small=True)
    check_attention(call(), reference())
    assert tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_shared_on_copies_and_behind_the_groups(kind):
    # each sequence has its prefix on pages of its own; two sequences are in no group
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, 64, "bf16", kind, 16, "token", 1, [3, 2, 1, 1], [70, 40, 0, 0],
                                                          [1, 9, 30, 2, 2, 50, 80], seed=3, copies=True)
    out, lse = call(off=off[:3].contiguous(), pl=pl[:2].contiguous())
    check_attention((out, lse), reference())
    out, lse = call(off=off[:1].contiguous(), pl=pl[:0].contiguous())  # no group at all
    check_attention((out, lse), reference())
    assert tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("kind, n", [("bf16", 1), ("bf16", 3), ("f16", 17), ("i8", 1), ("i8", 6), ("e4m3", 1)])
def test_sequences_shorter_than_the_prefix(kind, n):
    # the group's first one too; some see part of the prefix, or none of it
    import torch
    typ = "f16" if kind == "f16" else "bf16"
    lens = [0, 300, 299 + n, 5, 298 + n, 0, 500, 301, 1]
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, 64, typ, kind, 16, "token", n, [9], [300], [1] * 9, seed=4, lens=lens)
    out, lse = call()
    check_attention((out, lse), reference())
    assert tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_long_prefixes_and_many_groups(kind):
    # one prefix over the whole GPU; rows that fill several tiles; more groups than threads
    import torch
    for args in ((4, 1, 128, "bf16", kind, 64, "token", 1, [3], [20_000], [3, 300, 1]),
                 (4, 2, 64, "bf16", kind, 16, "head", 1, [150], [700], [1 + i % 9 for i in range(150)]),
                 (2, 1, 64, "bf16", kind, 16, "token", 1, [3] * 600, [17 + i % 40 for i in range(600)], [1 + i % 5 for i in range(1800)])):
        tg, cfg, c, q, off, pl, lens, reference, call = setup(*args, seed=5)
        out, lse = call()
        check_attention((out, lse), reference())
        assert tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_offsets_out_of_order_share_nothing(kind):
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(4, 2, 64, "bf16", kind, 16, "token", 1, [3, 3], [70, 40], [1, 9, 30, 2, 2, 7], seed=6)
    want = reference()
    call()
    for o, p in (([0, 4, 3], [70, 40]), ([0, 3, 7], [70, 40]), ([1, 3, 6], [70, 40]), ([-1, 3, 6], [70, 40]), ([0, 3, 6], [-1, 40]),
                 ([0, 3, 6], [70, 2 ** 30]), ([0, 3, 2 ** 40], [70, 40]), ([0, 3, 2 ** 32], [70, 40])):
        out, lse = call(off=ids(o, np.int64), pl=ids(p, np.int32))
        torch.cuda.synchronize()
        check_attention((out, lse), want)
        assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_ROW
        tg.tg_attn_clear_status(cfg)
    bad = lens.copy()
    bad[4] = 2 ** 30  # a length past the table: an empty sequence, as in a step
    out, lse = call(lens=bad)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_ROW
    bad[4] = 0
    check_attention((out, lse), reference(lens=bad))


@pytest.mark.parametrize("kind, n", [("bf16", 1), ("i8", 1), ("e4m3", 1), ("bf16", 9)])
def test_bad_pages_of_a_prefix(kind, n):
    # left out for the whole group, and flagged
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(4, 1, 64, "bf16", kind, 16, "token", n, [4, 2], [300, 90],
                                                          [n, n + 9, n + 30, n + 2, n, n + 8], seed=7)
    table = c.table_now()
    table[:4, 1] = 10 ** 6   # keys 16 .. 31 of the first group
    table[4:, 0] = -3        # keys 0 .. 15 of the second
    out, lse = call(table=table)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_PAGE
    for x in (c.keys, c.values):
        for b in range(6):
            x[b] = np.delete(x[b], np.s_[16:32] if b < 4 else np.s_[0:16], axis=0)
    check_attention((out, lse), reference(lens=lens - 16))


def test_numbers_behind_the_ends_and_neighbours_do_not_reach_a_row():
    # unused places hold NaN from the start; here a neighbour's queries and own keys do too
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, 64, "bf16", "bf16", 16, "token", 1, [3, 3], [100, 100],
                                                          [4, 9, 40, 5, 1, 0], seed=8)
    want = reference()
    out, lse = call()
    check_attention((out, lse), want)
    q[1] = float("nan")
    own = c.table[2, 7:9]
    c.v[ids(own, np.int64)] = float("inf")
    o2, z2 = call()
    # the group without them keeps its bits; a neighbour in the group may be computed another way
    for b in (3, 4, 5):
        assert torch.equal(o2[b], out[b]) and torch.equal(z2[b], lse[b])
    check_attention((o2[:1], z2[:1]), [x[:1] for x in want])
    assert o2[1].isnan().all() and not torch.isfinite(o2[2]).any()


@pytest.mark.parametrize("kind, n", [("bf16", 1), ("f16", 5), ("e4m3", 1), ("i8", 1), ("i8", 6), ("bf16", 40)])
def test_rows_beside_an_infinity_or_nan(kind, n):
    # among one sequence's own values: the others of its group, which share products with it, are as before;
    # in the prefix: all of the group's are not numbers
    import torch
    if n > 32:
        n, H = 32, 20  # a sequence's rows fill several tiles
    else:
        H = 8
    typ = "f16" if kind == "f16" else "bf16"
    own = [n + 3, n + 40, n + 1, n + 200]
    tg, cfg, c, q, off, pl, lens, reference, call = setup(H, 2, 64, typ, kind, 16, "token", n, [4], [150], own, seed=13)
    want = reference()
    page, slot = int(c.table[1, 155 // 16]), 155 % 16  # a key of sequence 1's own that all its tokens see
    if kind == "i8":
        parts(c.v, 2, 64, 16, "token")[1][page, 1, slot] = float("nan")
    elif kind == "e4m3":
        c.v.view(torch.uint8)[page, slot, 1, 5] = 0x7f
    else:
        c.v[page, slot, 1, 5] = float("inf")
    out, lse = call()
    others = [0, 2, 3]
    check_attention((out[others], lse[others]), [x[others] for x in want])
    assert not torch.isfinite(out[1, :, H // 2:]).all(-1).any() and torch.isfinite(out[1, :, :H // 2]).all()
    page, slot = int(c.table[0, 3]), 2
    if kind == "i8":
        parts(c.k, 2, 64, 16, "token")[1][page, 0, slot] = float("nan")
    elif kind == "e4m3":
        c.k.view(torch.uint8)[page, slot, 0, 0] = 0x7f
    else:
        c.k[page, slot, 0, 0] = float("nan")
    out, lse = call()
    assert out[:, :, :H // 2].isnan().all() and lse[:, :, :H // 2].isnan().all()


def test_peaked_weights_of_prefix_or_own():
    # all the weight on one side: the other adds nothing, and nothing overflows
    import torch
    for kind in ("bf16", "i8", "f16"):
        typ = "f16" if kind == "f16" else "bf16"
        tg, cfg, c, q, off, pl, lens, reference, call = setup(4, 1, 64, typ, kind, 16, "token", 1, [4], [256], [30, 40, 50, 60], seed=9)
        # the row's query along one key: of the prefix for two sequences, its own for the others
        for b, j in ((0, 17), (1, 255), (2, 256), (3, 300)):
            q[b, 0] = torch.from_numpy(c.keys[b][j, 0] * 12).to(q)
        out, lse = call()
        check_attention((out, lse), reference())


@pytest.mark.parametrize("kind, n", [("bf16", 1), ("i8", 1), ("bf16", 7)])
def test_stream_and_graph_follow_the_lengths(kind, n):
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, 128, "bf16", kind, 16, "head", n, [4, 4, 1], [300, 64, 9],
                                                          [n, n + 50, n + 3, n, n + 1, n + 20, n + 9, n, n + 30], seed=10)
    want = reference()
    out, lse = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, z2 = call(stream=side)
    side.synchronize()
    assert torch.equal(o2, out) and torch.equal(z2, lse)
    kl, table = ids(lens, np.int32), c.table_now()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(o2, z2, table=table, lens=kl)
    for now, p in ((lens, [300, 64, 9]), ([300, 340, 20, 301, 64, 70, 70, 10, 39], [299, 30, 0]), (lens, [0, 0, 0]), (lens, [300, 64, 9])):
        now = np.minimum(now, lens)
        kl.copy_(ids(now, np.int32))
        pl.copy_(ids(p, np.int32))
        g.replay()
        torch.cuda.synchronize()
        check_attention((o2, z2), reference(lens=now))
    assert torch.equal(o2, out) and torch.equal(z2, lse)
    assert tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("kind, n", [("bf16", 1), ("i8", 1), ("e4m3", 1), ("bf16", 9), ("i8", 9)])
def test_after_waits_ran_out(kind, n):
    import torch
    from tests.test_gpu_attention_timeout import run_out
    tg, cfg, c, q, off, pl, lens, reference, call = setup(12, 3, 128, "bf16", kind, 16, "token", n, [5, 3], [2000, 300],
                                                          [n + 3 * i for i in range(8)], seed=11)
    out, table, kl = torch.empty_like(q), c.table_now(), ids(lens, np.int32)
    lse = torch.empty(q.shape[:3], device="cuda")
    run_out(cfg, lambda: call(out, lse, table=table, lens=kl), out)


def test_refusals():
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(4, 2, 64, "bf16", "bf16", 16, "token", 1, [3, 2], [70, 40], [1, 9, 30, 2, 2], seed=12)
    small = tg.AttnConfig(num_heads=4, num_kv_heads=2, head_dim=64, max_shared_tokens=4)
    none = tg.AttnConfig(num_heads=4, num_kv_heads=2, head_dim=64)
    out = torch.empty_like(q)
    for cfg2 in (small, none):
        with pytest.raises((tg.TGError, ValueError)):
            tg.tg_attend_shared(q, ids(lens, np.int32), c.device_table(), c.k, c.v, off, pl, cfg2, out)
    for kw in (dict(off=off[:2].contiguous()), dict(off=off.int()), dict(pl=pl.long()), dict(pl=pl.cpu())):
        with pytest.raises((tg.TGError, ValueError)):
            call(**kw)


@pytest.mark.parametrize("kind, n, typ", [("bf16", 1, "bf16"), ("f16", 1, "f16"), ("e4m3", 1, "f16"), ("i8", 1, "bf16"), ("i8", 9, "f16")])
@pytest.mark.parametrize("rise", [0.5, 4.0])
def test_scores_that_rise_inside_a_tile(kind, n, typ, rise):
    # every key scores above the one before: references rise in each tile, what came before is scaled down
    import torch
    D, L, own = 64, 300, [n + 40, n + 3, n + 150]
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, D, typ, kind, 16, "token", n, [3], [L], own, seed=14)
    u = np.random.default_rng(1).choice([-1.0, 1.0], D)
    q.copy_(torch.from_numpy(np.broadcast_to(u, q.shape).copy()).to(q))
    for b in range(3):
        for j in range(int(lens[b])):
            if b and j < L:
                continue  # (the shared pages, or copies of the first one's)
            k = u * (j % 400) * rise / D
            page, slot = int(c.table[b, j // 16]), j % 16
            if kind == "i8":
                codes, scales = parts(c.k, 2, D, 16, "token")
                codes[page, slot] = torch.from_numpy((128 + 127 * u).astype(np.uint8)).cuda()
                s = np.float32((j % 400) * rise / D / 127)
                scales[page, :, slot] = float(s)
                c.keys[b][j] = u * 127 * np.float64(s)
            else:
                row = torch.from_numpy(np.broadcast_to(k * (10 if kind == "e4m3" else 1), (2, D)).astype(np.float32)).cuda().to(c.k.dtype)
                c.k.view(torch.uint8 if kind == "e4m3" else c.k.dtype)[page, slot] = row.view(torch.uint8) if kind == "e4m3" else row
                c.keys[b][j] = f64(row)
    for b in (1, 2):
        whole = L // 16 * 16
        c.keys[b][:L] = c.keys[0][:L]
        for j in range(whole, L):  # (the page in which the prefix ends is each one's copy)
            dst, src = int(c.table[b, j // 16]), int(c.table[0, j // 16])
            if kind == "i8":
                codes, scales = parts(c.k, 2, D, 16, "token")
                codes[dst, j % 16] = codes[src, j % 16]
                scales[dst, :, j % 16] = scales[src, :, j % 16]
            else:
                raw = c.k.view(torch.uint8) if kind == "e4m3" else c.k
                raw[dst, j % 16] = raw[src, j % 16]
    out, lse = call()
    check_attention((out, lse), reference())
    o2, z2 = torch.empty_like(out), torch.empty_like(lse)
    tg.tg_attend_step(q, ids(lens, np.int32), c.device_table(), c.k, c.v, cfg, o2, z2)
    check_attention((o2, z2), reference())


def test_a_key_head_for_every_query_head_and_more_sequences_than_a_tile():
    for kind in ("bf16", "i8"):
        tg, cfg, c, q, off, pl, lens, reference, call = setup(3, 3, 64, "bf16", kind, 16, "head", 1, [100, 70], [200, 40],
                                                              [i % 11 for i in range(170)], seed=15)
        check_attention(call(), reference())


def test_more_sequences_than_the_layout_holds():
    # read one by one
    B = 18000
    tg, cfg, c, q, off, pl, lens, reference, call = setup(2, 1, 16, "f16", "f16", 16, "token", 1, [B // 2, B // 2], [20, 16],
                                                          [1 + i % 3 for i in range(B)], seed=16)
    check_attention(call(), reference())
