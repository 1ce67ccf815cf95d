"""Over an i8 cache a row is as exact as the keys that it sees allow: values of later tokens, of neighbours in a
shared tile and of a prefix that it is too short for may be larger by any factor."""
import numpy as np
import pytest

from oracle import attention_oracle as A
from tests.attention_util import check_attention, f64, ids, torch_types
from tests.quant_util import I8Cache, parts
from tests.test_gpu_attention_shared import setup

pytestmark = pytest.mark.gpu


def seen_reference(c, q, n, rep, kind, lens=None):
    """Rows of [B, n, H] and what they may be off by.

    A weight times its value's scale is rounded to f16 in a unit of which the row's largest such product is 2^5 at least
    (2^8 in the step kernel): 2^-11 of itself, or half of f16's smallest step, 2^-25, which is 2^-30 of that largest product,
    and its code is 127 at most (127 scales: the largest magnitude of the key's values).  Inside a tile of 128 keys a product may be scaled three
    times more, each a rounding."""
    B, _, H, D = q.shape
    lens = c.lens if lens is None else np.asarray(lens)
    res = [np.zeros((B, n, H, D)), np.zeros((B, n, H, D)), np.zeros((B, n, H)), np.zeros((B, n, H))]
    scale = 1 / np.sqrt(D)
    for b in range(B):
        for h in range(H):
            k, v = c.keys[b][:, h // rep], c.values[b][:, h // rep]
            sees = int(lens[b]) - n + 1 + np.arange(n)
            o, tol, z, ztol = A.attend(q[b, :, h], k, v, sees, scale, kind, "f16")
            for j in range(n):
                m = min(max(int(sees[j]), 0), len(k))
                if m:
                    s = k[:m] @ q[b, j, h] * scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    tol[j] += 3 * 2.0 ** -11 * (w @ np.abs(v[:m])) + m * 2.0 ** -30 * (w * np.abs(v[:m]).max(-1)).max()
            for dst, x in zip(res, (o, tol, z, ztol)):
                dst[b, :, h] = x
    return res


def enlarge(c, heads, dim, b, pos, factor):
    """Multiply the value scales of sequence b's tokens at pos (and what the cache stands for) by a power of two (in two
    factors that f32 holds)."""
    scales = parts(c.v, heads, dim, c.page, c.layout)[1]
    pos = np.asarray(pos, np.int64)
    if len(pos):
        first = min(factor, 2.0 ** 100)
        for f in (first, factor / first if factor else 0.0):
            scales[ids(c.table[b, pos // c.page], np.int64), :, ids(pos % c.page, np.int64)] *= f
        c.values[b] = c.values[b].copy()
        c.values[b][pos] *= factor


STEPS = [
    # heads, key heads, dim, type, page, layout, n: up to 8 rows, 16, the tensor-memory kernel, rows over small pages
    (8, 2, 128, "bf16", 16, "token", 2), (8, 2, 64, "f16", 32, "head", 4), (8, 2, 128, "bf16", 16, "token", 6),
    (8, 2, 64, "f16", 64, "head", 17), (4, 1, 64, "f16", 4, "token", 9), (5, 5, 80, "bf16", 2, "head", 30),
    (16, 1, 128, "f16", 8, "token", 5),
]


@pytest.mark.parametrize("how", ["last", "largest", "rising"])
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_later_tokens_of_a_step(case, how):
    # the last token's values are larger by 2^25 or 2^100; each token's by 2^12 than the one's before
    import torch
    import logits_processing_token_gb300 as tg
    H, G, D, typ, page, layout, n = case
    lens = [n, n + 1, 126 + n, 128 + n, 500, max(n - 1, 1)]
    c = I8Cache(lens, G, D, page, layout, 21)
    for b, L in enumerate(lens):
        if how == "rising":
            for j in range(min(n, L)):
                enlarge(c, G, D, b, [L - min(n, L) + j], 2.0 ** min(12 * j, 96))
        else:
            enlarge(c, G, D, b, [L - 1], 2.0 ** (25 if how == "last" else 100))
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype="i8", page_size=page, page_layout=layout,
                        max_step_tokens=32)
    q = torch.from_numpy(np.random.default_rng(22).normal(0, 2, (len(lens), n, H, D)).astype(np.float32)).cuda().to(torch_types()[typ])
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
    tg.tg_attend_step(q, ids(lens, np.int32), c.device_table(), c.k, c.v, cfg, out, lse)
    want = seen_reference(c, f64(q), n, H // G, typ)
    if typ == "f16":  # results past f16's end are infinite
        big = np.abs(want[0]) + want[1] > 65000
        out, want[0] = torch.where(torch.from_numpy(big).cuda(), 0.0, out.float()), np.where(big, 0.0, want[0])
    check_attention((out, lse), want)
    assert tg.tg_attn_status_word(cfg) == 0


def check_shared(s, n, rep, typ):
    tg, cfg, c, q, off, pl, lens, reference, call = s
    out, lse = call()
    check_attention((out, lse), seen_reference(c, f64(q), n, rep, typ, lens))
    return out, lse


@pytest.mark.parametrize("n", [2, 6])
def test_later_tokens_of_a_shared_call(n):
    s = setup(16, 4, 64, "bf16", "i8", 16, "token", n, [4, 2], [200, 64], [n, n + 9, n + 130, n + 300, n, n + 1], seed=51)
    for b, L in enumerate(s[6]):
        enlarge(s[2], 4, 64, b, [L - 1], 2.0 ** 25)
    check_shared(s, n, 4, "bf16")


@pytest.mark.parametrize("gone", [False, True])
@pytest.mark.parametrize("n", [1, 3])
def test_a_first_own_tile_without_values(n, gone):
    # behind a neighbour whose values are 2^30 times as large: a tile of values that are 0, or on pages that do not exist
    # (so many groups that a CTA has several of a group's sequences)
    groups = 120
    tg, cfg, c, q, off, pl, lens, reference, call = setup(4, 2, 64, "bf16", "i8", 16, "token", n, [4] * groups, [64] * groups,
                                                          [300, 500, 400, 150] * groups, seed=52)
    for b in range(4 * groups):
        if b % 2 == 0:
            enlarge(c, 2, 64, b, np.arange(64, lens[b]), 2.0 ** 30)
        elif not gone:
            enlarge(c, 2, 64, b, np.arange(64, min(64 + 128, lens[b] - n)), 0.0)
        else:
            end = 12 if b % 4 == 1 else 8
            c.table[b, 4:end] = -7
            for x in (c.keys, c.values):
                x[b] = np.delete(x[b], np.s_[64:16 * end], axis=0)
    out, lse = call()
    want = seen_reference(c, f64(q), n, 2, "bf16", [len(k) for k in c.keys])
    check_attention((out, lse), want)
    assert tg.tg_attn_status_word(cfg) == (tg.TG_FLAG_BAD_PAGE if gone else 0)


@pytest.mark.parametrize("n", [1, 6])
def test_a_prefix_that_a_sequence_is_too_short_for(n):
    # its end's values are 2^40 times as large; a shorter sequence of the group has none of those
    groups = 100
    lens = [420, 200, 300 + n, 250] * groups
    s = setup(4, 2, 128, "bf16", "i8", 16, "token", n, [4] * groups, [304] * groups, [1] * (4 * groups), seed=53, lens=lens)
    c = s[2]
    scales = parts(c.v, 2, 128, 16, "token")[1]
    for b in range(0, 4 * groups, 4):
        scales[ids(c.table[b, 256 // 16:304 // 16], np.int64)] *= 2.0 ** 40
    for b, L in enumerate(lens):
        on = [p for p in range(256, min(304, L)) if c.table[b, p // 16] == c.table[b // 4 * 4, p // 16]]
        c.values[b] = c.values[b].copy()
        c.values[b][on] *= 2.0 ** 40
    check_shared(s, n, 2, "bf16")


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("first", [False, True])
def test_neighbours_farther_apart_than_numbers_reach(n, first):
    # values of 2^-60 and of 2^90 in one tile, in either order
    s = setup(16, 4, 64, "bf16", "i8", 16, "token", n, [6], [32], [n + 40, n, n + 200, n + 9, n + 3, n + 150], seed=54)
    tg, cfg, c, q, off, pl, lens, reference, call = s
    scales = parts(c.v, 4, 64, 16, "token")[1]
    scales *= 2.0 ** -60
    for b in range(6):
        c.values[b] = c.values[b] * 2.0 ** -60
        if (b % 2 == 0) == first:
            enlarge(c, 4, 64, b, np.arange(32, lens[b]), 2.0 ** 150)
    check_shared(s, n, 4, "bf16")


@pytest.mark.parametrize("n", [1, 6])
def test_a_neighbours_nan_scales(n):
    # of values and of keys: only the sequence that sees them comes out so
    import torch
    tg, cfg, c, q, off, pl, lens, reference, call = s = setup(8, 2, 64, "bf16", "i8", 16, "token", n, [5], [100],
                                                              [n + 30, n + 150, n + 1, n, n + 60], seed=55)
    want = seen_reference(c, f64(q), n, 4, "bf16", lens)
    for pool, b, key in ((c.v, 1, 130), (c.k, 4, 120)):
        parts(pool, 2, 64, 16, "token")[1][int(c.table[b, key // 16]), :, key % 16] = float("nan")
    out, lse = call()
    keep = [0, 2, 3]
    check_attention((out[keep], lse[keep]), [x[keep] for x in want])
    assert out[[1, 4]].isnan().all() and lse[4].isnan().all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_a_rows_bits_are_its_own_keys(case):
    # with the last token's values and keys larger, the tokens before it keep their bits
    import torch
    import logits_processing_token_gb300 as tg
    H, G, D, typ, page, layout, n = case
    lens = [n, n + 130, 500, 1]
    c = I8Cache(lens, G, D, page, layout, 23)
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype="i8", page_size=page, page_layout=layout,
                        max_step_tokens=32)
    q = torch.from_numpy(np.random.default_rng(24).normal(0, 2, (len(lens), n, H, D)).astype(np.float32)).cuda().to(torch_types()[typ])
    got = []
    for factor in (1.0, 2.0 ** 90):
        for b, L in enumerate(lens):
            enlarge(c, G, D, b, [L - 1], factor)
            parts(c.k, G, D, page, layout)[1][int(c.table[b, (L - 1) // page]), :, (L - 1) % page] *= min(factor, 64.0)
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
        tg.tg_attend_step(q, ids(lens, np.int32), c.device_table(), c.k, c.v, cfg, out, lse)
        got.append((out[:, :-1], lse[:, :-1]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("n", [1, 6])
def test_a_sequences_bits_are_its_own_keys_in_a_shared_call(n):
    import torch
    groups = 60
    tg, cfg, c, q, off, pl, lens, reference, call = setup(16, 4, 64, "bf16", "i8", 16, "token", n, [4] * groups, [200] * groups,
                                                          [n, n + 9, n + 130, n + 300] * groups, seed=56)
    got = [call()]
    for b in range(0, len(lens), 2):
        enlarge(c, 4, 64, b, np.arange(200, lens[b]), 2.0 ** 50)
    got.append(call())
    odd = list(range(1, len(lens), 2))
    assert torch.equal(got[0][0][odd], got[1][0][odd]) and torch.equal(got[0][1][odd], got[1][1][odd])
