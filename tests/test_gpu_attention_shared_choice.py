"""Where tg_attend_shared is a step: nothing that a row tile could share, or as many groups as sequences.
The results are the step's to the bit, and neither the groups' offsets nor their prefixes are read."""
import numpy as np
import pytest

from tests.attention_util import check_attention, ids
from tests.test_gpu_attention_shared import setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind, H, G, n, members", [
    ("bf16", 8, 2, 17, [3, 2]),      # 68 rows a sequence: one to a tile of 128
    ("i8", 8, 2, 17, [3, 2]), ("e4m3", 20, 2, 7, [4]),
    ("f16", 40, 1, 2, [3]), ("i8", 66, 1, 1, [4]),
    ("bf16", 20, 1, 32, [3]),        # a sequence's rows fill several tiles
    ("bf16", 8, 2, 6, [1, 1, 1, 1]), ("i8", 8, 2, 6, [4, 0, 0, 0]), ("bf16", 8, 2, 1, [3, 1, 0, 0]),
])
def test_calls_that_are_steps(kind, H, G, n, members):
    import torch
    typ = "f16" if kind == "f16" else "bf16"
    own = [n + 13 * i for i in range(sum(members))]
    tg, cfg, c, q, off, pl, lens, reference, call = setup(H, G, 64, typ, kind, 16, "token", n, members, [90] * len(members), own, seed=61)
    table = c.table_now()
    out, lse = call(table=table)
    check_attention((out, lse), reference())
    o2, z2 = torch.empty_like(out), torch.empty_like(lse)
    tg.tg_attend_step(q, ids(lens, np.int32), table, c.k, c.v, cfg, o2, z2)
    assert torch.equal(out, o2) and torch.equal(lse, z2)
    call(table=table, off=torch.full_like(off, -1), pl=torch.full_like(pl, -1))
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == 0


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
def test_two_sequences_to_a_tile_share(kind):
    # 64 rows each: the offsets are read, and refused where they are out of order
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = setup(8, 2, 64, "bf16", kind, 16, "token", 16, [3, 2], [90, 40],
                                                          [16, 40, 300, 17, 20], seed=62)
    check_attention(call(), reference())
    assert tg.tg_attn_status_word(cfg) == 0
    check_attention(call(off=ids([0, 4, 3], np.int64)), reference())
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_ROW
