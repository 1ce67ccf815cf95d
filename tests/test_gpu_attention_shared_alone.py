"""Rows of a shared call that are computed again, because a neighbour's values are no numbers: over many keys,
past pages that do not exist, in every kind of cache; and rows that are lost themselves cost no such walk."""
import numpy as np
import pytest

from tests.attention_util import check_attention, ids
from tests.test_gpu_attention_shared import setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind, typ, H, G, D, page, layout, n", [
    ("bf16", "bf16", 8, 2, 128, 16, "token", 1), ("f16", "f16", 6, 3, 80, 8, "head", 4), ("bf16", "bf16", 5, 1, 16, 256, "token", 3),
    ("e4m3", "bf16", 8, 2, 64, 32, "head", 1), ("e4m3", "f16", 3, 3, 112, 16, "token", 6), ("f16", "f16", 20, 1, 96, 1024, "head", 2)])
def test_rows_computed_again(kind, typ, H, G, D, page, layout, n):
    import torch
    own = [n + 3, n + 300, n, n + 31, n + 64]
    tg, cfg, c, q, off, pl, lens, reference, call = setup(H, G, D, typ, kind, page, layout, n, [5], [1100], own, seed=71)
    table = c.table_now()
    if page <= 32:  # a page of the prefix that is not there, for all
        lost = np.s_[9 * page:10 * page]
        table[:, 9] = 10 ** 6
        for x in (c.keys, c.values):
            for b in range(5):
                x[b] = np.delete(x[b], lost, axis=0)
    want = reference(lens=[len(k) for k in c.keys])
    key = 1100 + 290  # of sequence 1's own, seen by all its tokens
    where, slot = int(c.table[1, key // page]), key % page
    bad = (where, slot) if layout == "token" else (where, slice(None), slot)
    if kind == "e4m3":
        c.v.view(torch.uint8)[bad] = 0x7f
    else:
        c.v[bad] = float("-inf")
    out, lse = call(table=table)
    rest = [0, 2, 3, 4]
    check_attention((out[rest], lse[rest]), [x[rest] for x in want])
    assert not torch.isfinite(out[1].float()).any() and torch.isfinite(lse[1]).all()
    o2, z2 = call(table=table)
    assert torch.equal(o2[rest], out[rest]) and torch.equal(z2, lse)
    assert tg.tg_attn_status_word(cfg) == (tg.TG_FLAG_BAD_PAGE if page <= 32 else 0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_a_lost_prefix_costs_no_walk(kind):
    # a key that is no number at the beginning of a prefix of 30,000: every row is NaN (18 ms where each walked all keys)
    import torch
    from tests.quant_util import parts
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, 128, "bf16", kind, 64, "token", 1, [8], [30_000], [5 + i for i in range(8)], seed=72)
    page = int(c.table[0, 0])
    if kind == "i8":
        parts(c.k, 2, 128, 64, "token")[1][page, :, 7] = float("nan")
    elif kind == "e4m3":
        c.k.view(torch.uint8)[page, 7] = 0x7f
    else:
        c.k[page, 7] = float("nan")
    table, kl = c.table_now(), ids(lens, np.int32)
    out, lse = call(table=table, lens=kl)
    assert out.isnan().all() and lse.isnan().all()
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call(out, lse, table=table, lens=kl)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    assert min(times) < 5.0
