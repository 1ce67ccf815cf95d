"""Steps of many rows over 8-bit caches and shared calls at the ends of what they take: pages longer
than a tile, small heads, strided queries, outputs off a 32-byte boundary, a sequence named twice,
two handles at once."""
import numpy as np
import pytest

from tests.attention_util import check_attention, ids
from tests.test_gpu_attention_i8 import run_step
from tests.test_gpu_attention_shared import setup
from tests.test_gpu_attention_step import run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind, typ, D, page, layout, n", [
    ("bf16", "bf16", 64, 256, "token", 1), ("i8", "bf16", 128, 1024, "head", 1), ("e4m3", "f16", 32, 512, "token", 1),
    ("i8", "f16", 16, 256, "token", 6), ("f16", "f16", 112, 1024, "head", 6)])
def test_pages_longer_than_a_tile(kind, typ, D, page, layout, n):
    # prefixes that end in a tile, at its end and at a page's; own keys on the prefix's last page
    own = [n, n + 1, 130, 200, n, 1200, n]
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, D, typ, kind, page, layout, n, [4, 3], [1100, 128], own, seed=41)
    check_attention(call(), reference())
    assert tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("case", [
    (4, 1, 16, "bf16", "e4m3", 8, "token", 9, [9, 8, 0, 200]),
    (9, 3, 48, "f16", "e4m3", 1024, "head", 7, [1300, 7]),
    (20, 1, 128, "bf16", "e4m3", 16, "token", 1, [129, 1, 0, 2000]),
    (40, 2, 80, "f16", "e4m3", 64, "token", 30, [31, 400]),
], ids=lambda c: "-".join(map(str, c[:8])))
def test_many_rows_over_e4m3(case):
    run_case(*case, seed=42)


@pytest.mark.parametrize("case", [
    (6, 2, 32, "f16", 1024, "token", 9, [1500, 9, 0]),
    (17, 1, 16, "bf16", 8, "head", 1, [1, 0, 127, 128, 129]),
    (40, 2, 112, "f16", 256, "token", 30, [31, 400]),
], ids=lambda c: "-".join(map(str, c[:7])))
def test_many_rows_over_i8(case):
    run_step(*case, seed=43)


@pytest.mark.parametrize("kind, n", [("bf16", 1), ("i8", 1), ("e4m3", 5), ("bf16", 5)])
def test_strided_queries_and_outputs_off_32_bytes(kind, n):
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, 80, "bf16", kind, 16, "token", n, [3, 2], [300, 47],
                                                          [n, n + 30, 150, n, n], seed=44)
    B, _, H, D = q.shape
    wide = torch.full((B * n, 2 * H * D + 8), float("nan"), device="cuda", dtype=q.dtype)
    qs = wide[:, 8:8 + H * D].unflatten(1, (H, D))
    qs.copy_(q.reshape(B * n, H, D))
    room = torch.full((B * n * H * D + 24,), 7.0, device="cuda", dtype=q.dtype)
    at = next(x for x in range(0, 24, 8) if (room.data_ptr() + 2 * x) % 32 == 16)
    out = room[at:at + B * n * H * D].view(B, n, H, D)
    lse = torch.empty(B, n, H, device="cuda")
    tg.tg_attend_shared(qs.view(B, n, H, D) if n == 1 else qs.unflatten(0, (B, n)), ids(lens, np.int32), c.table_now(), c.k, c.v, off, pl, cfg, out, lse)
    check_attention((out, lse), reference())
    assert (room[:at] == 7).all() and (room[at + out.numel():] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_a_sequence_named_twice(kind):
    # the same row of the table and the same length twice in a group, and once behind it
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, 64, "bf16", kind, 16, "token", 1, [2, 1], [70, 0], [30, 30, 100], seed=45)
    c.table[1, :], c.table[2, :] = c.table[0, :], c.table[0, :]
    lens = np.asarray([100, 100, 100])
    for x in (c.keys, c.values):
        x[1] = x[2] = x[0]
    c.lens = lens
    check_attention(call(lens=lens), reference(lens))


def test_two_handles_at_once():
    import torch
    made = [setup(8, 2, 128, "bf16", kind, 16, "token", n, [4, 4], [2000, 1500], [n + 40 * i for i in range(8)], seed=46 + n)
            for kind, n in (("bf16", 1), ("i8", 5))]
    tables = [m[2].table_now() for m in made]
    lens = [ids(m[6], np.int32) for m in made]
    want = [m[8](table=t, lens=l) for m, t, l in zip(made, tables, lens)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[] for _ in made]
    for _ in range(10):
        for i, m in enumerate(made):
            with torch.cuda.stream(streams[i]):
                got[i].append(m[8](table=tables[i], lens=lens[i], stream=streams[i]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for o, z in g:
            assert torch.equal(o, w[0]) and torch.equal(z, w[1])
    assert all(m[0].tg_attn_status_word(m[1]) == 0 for m in made)


@pytest.mark.parametrize("kind, n", [("bf16", 1), ("i8", 1), ("e4m3", 5), ("f16", 30)])
def test_slots_that_name_no_page(kind, n):
    # empty slots at a group's beginning, in it and at its end; sequences shorter than the prefix; a group of such ones
    # alone; more sequences than a row tile holds: their rows of the table name the pages of their own lengths only
    typ = "f16" if kind == "f16" else "bf16"
    first = [0, 40, 0, 300 + n, 299 + n, 310, 0, 298 + n]
    lens = first + [0, 20, 0] + ([0] * 70 + [200 + n, 260, 0] if n == 1 else [0])
    members = [len(first), 3, len(lens) - len(first) - 3]
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, 64, typ, kind, 16, "token", n, members, [300, 64, 200], [1] * len(lens), seed=47,
                                                          lens=lens)
    for b, m in enumerate(lens):
        c.table[b, -(-int(m) // 16):] = -1
    check_attention(call(), reference())
    assert tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("n, ratio", [(1, 2.0 ** 12), (1, 2.0 ** 30), (6, 2.0 ** 20), (1, 2.0 ** 110)])
def test_i8_values_far_larger_in_another_sequence(n, ratio):
    # every other sequence's own values are larger by a factor that f16 weights cannot hold: the others, whose rows
    # share its tiles, are as exact as by themselves (their tolerances know their own values only)
    import torch
    from tests.quant_util import parts
    H, G = (16, 8) if n == 1 else (8, 4)
    tg, cfg, c, q, off, pl, lens, reference, call = setup(H, G, 64, "bf16", "i8", 16, "token", n, [24, 6], [208, 64], [n + 5 * (i % 7) for i in range(30)],
                                                          seed=48)
    pre = np.repeat([208, 64], [24, 6])
    scales = parts(c.v, G, 64, 16, "token")[1]
    for b in range(1, 30, 2):
        j = np.arange(pre[b], lens[b])
        scales[ids(c.table[b, j // 16], np.int64), :, ids(j % 16, np.int64)] *= ratio
        c.values[b] = c.values[b].copy()
        c.values[b][pre[b]:] *= ratio
    out, lse = call()
    with np.errstate(over="ignore"):
        want = reference()
    even = list(range(0, 30, 2))
    check_attention((out[even], lse[even]), [x[even] for x in want])
    odd = list(range(1, 30, 2))
    check_attention((out[odd], lse[odd]), [x[odd] for x in want])
    assert tg.tg_attn_status_word(cfg) == 0
