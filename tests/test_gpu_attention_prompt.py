"""tg_attend_prompt against the 64-bit oracle: packed sequences of any length,
empty ones, more queries than keys, strides, tiles that end in another sequence."""
import numpy as np
import pytest

from oracle import attention_oracle as A
from tests.attention_util import check_attention, f64, ids, torch_types

pytestmark = pytest.mark.gpu

CASES = [
    # heads, key heads, dim, type, causal, query lengths, key lengths (None: the same)
    (2, 1, 128, "bf16", True, [1], None),
    (2, 2, 64, "f16", True, [61], None),
    (4, 2, 128, "bf16", True, [1, 2, 0, 63, 64, 65, 127, 128, 129, 255, 256, 257], None),
    (4, 1, 64, "bf16", True, [300, 0, 5, 513], None),
    (3, 3, 80, "f16", True, [130, 40], None),
    (2, 1, 96, "bf16", False, [70, 200], None),
    (2, 1, 16, "f16", True, [33, 290], None),
    (4, 4, 128, "f16", False, [5, 260, 0], [300, 64, 7]),
    (4, 2, 128, "bf16", True, [40, 100, 7, 3], [400, 30, 0, 3]),
    (2, 1, 64, "f16", True, [500, 129], [130, 700]),
    (2, 1, 112, "bf16", False, [129, 3, 2], [0, 1, 513]),
    (8, 1, 128, "bf16", True, [700], None),
]


def reference(q, k, v, nq, nk, causal, scale, kind):
    T, H, D = q.shape
    G = k.shape[1]
    res = [np.zeros((T, H, D)), np.zeros((T, H, D)), np.zeros((T, H)), np.zeros((T, H))]
    a = b = 0
    for m, n in zip(nq, nk):
        sees = np.arange(m) + 1 + n - m if causal else np.full(m, n)
        for h in range(H):
            r = A.attend(q[a:a + m, h], k[b:b + n, h // (H // G)], v[b:b + n, h // (H // G)], sees, scale, kind)
            for dst, x in zip(res, r):
                dst[a:a + m, h] = x
        a, b = a + m, b + n
    return res


def make(H, G, D, typ, nq, nk, seed, pad=0, grow=1.0):
    import torch
    rng = np.random.default_rng(seed)
    t = torch_types()[typ]
    Tq, Tk = sum(nq), sum(nk)
    q = torch.from_numpy(rng.normal(0, 2 * grow, (Tq, H * D + 8 * pad)).astype(np.float32)).cuda().to(t)[:, :H * D].unflatten(1, (H, D))
    kv = torch.from_numpy(rng.normal(0, 1, (Tk, 2 * G * D + 8 * pad)).astype(np.float32)).cuda().to(t)
    k, v = kv[:, :G * D].unflatten(1, (G, D)), kv[:, G * D:2 * G * D].unflatten(1, (G, D))
    off = lambda n: ids(np.concatenate([[0], np.cumsum(n)]), np.int64)  # noqa: E731
    return q, k, v, off(nq), off(nk)


def run_case(H, G, D, typ, causal, nq, nk, seed=0, pad=0, with_lse=True, grow=1.0):
    import torch
    import logits_processing_token_gb300 as tg
    same = nk is None
    nk = nq if same else nk
    q, k, v, qo, ko = make(H, G, D, typ, nq, nk, seed, pad, grow)
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ)
    out = torch.full(q.shape, float("nan"), device="cuda", dtype=q.dtype)
    lse = torch.full(q.shape[:2], float("nan"), device="cuda") if with_lse else None
    tg.tg_attend_prompt(q, k, v, qo, None if same else ko, cfg, out, lse, causal=causal)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == 0
    check_attention((out, lse), reference(f64(q), f64(k), f64(v), nq, nk, causal, 1 / np.sqrt(D), typ))
    return cfg, q, k, v, qo, ko, out, lse


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])) + "-%dx%d" % (len(c[5]), max(c[5])))
def test_prompt_matches_oracle(case):
    run_case(*case)


def test_prompt_strides_no_lse_and_peaked_weights():
    run_case(4, 2, 128, "bf16", True, [200, 33], None, seed=1, pad=3, with_lse=False)
    run_case(4, 2, 64, "f16", True, [40, 333], [100, 333], seed=2, pad=1)
    run_case(4, 2, 128, "bf16", True, [200, 130], None, seed=3, grow=20.0)
    run_case(4, 2, 128, "f16", False, [200, 130], None, seed=4, grow=20.0)


def test_prompt_long():
    import torch
    import logits_processing_token_gb300 as tg
    # rows spread over a long prompt, against the oracle
    H, G, D, n = 2, 1, 128, 9001
    q, k, v, qo, ko = make(H, G, D, "bf16", [n], [n], 5)
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D)
    out, lse = torch.empty_like(q.contiguous()), torch.empty(q.shape[:2], device="cuda")
    tg.tg_attend_prompt(q, k, v, qo, None, cfg, out, lse)
    rows = np.unique(np.concatenate([np.arange(0, n, 451), [n - 1, n - 2, 128, 255, 256]]))
    for h in range(H):
        want = A.attend(f64(q)[rows, h], f64(k)[:, 0], f64(v)[:, 0], rows + 1, 1 / np.sqrt(D), "bf16")
        at = ids(rows, np.int64)
        check_attention((out[at, h], lse[at, h]), want)


def test_prompt_sequences_do_not_touch():
    # NaN and infinities in one sequence stay in it, whichever tiles it shares
    import torch
    import logits_processing_token_gb300 as tg
    for D, typ in ((128, "bf16"), (64, "f16"), (80, "bf16")):
        nq = [70, 90, 200]
        q, k, v, qo, ko = make(4, 2, D, typ, nq, nq, 6)
        cfg = tg.AttnConfig(num_heads=4, num_kv_heads=2, head_dim=D, dtype=typ)
        want = reference(f64(q), f64(k), f64(v), nq, nq, True, 1 / np.sqrt(D), typ)
        for t in (q, k, v):
            t[70:110] = float("nan")
            t[110:160] = float("inf")
        out, lse = torch.empty_like(q.contiguous()), torch.empty(q.shape[:2], device="cuda")
        tg.tg_attend_prompt(q, k, v, qo, None, cfg, out, lse)
        for a, b in ((0, 70), (160, 360)):
            check_attention((out[a:b], lse[a:b]), [x[a:b] for x in want])


def test_prompt_equal_bits_stream_and_graph():
    import torch
    import logits_processing_token_gb300 as tg
    cfg, q, k, v, qo, ko, out, lse = run_case(4, 2, 128, "bf16", True, [300, 10, 129], None, seed=7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, z2 = torch.empty_like(out), torch.empty_like(lse)
    with torch.cuda.stream(side):
        tg.tg_attend_prompt(q, k, v, qo, None, cfg, o2, z2)
    side.synchronize()
    assert torch.equal(o2, out) and torch.equal(z2, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tg.tg_attend_prompt(q, k, v, qo, None, cfg, o2, z2)
    nq = [129, 10, 300]
    qo.copy_(ids(np.concatenate([[0], np.cumsum(nq)]), np.int64))
    g.replay()
    torch.cuda.synchronize()
    check_attention((o2, z2), reference(f64(q), f64(k), f64(v), nq, nq, True, 1 / np.sqrt(128), "bf16"))


def test_prompt_bad_offsets_are_flagged():
    import torch
    import logits_processing_token_gb300 as tg
    nq = [100, 50, 80]
    cfg, q, k, v, qo, ko, out, lse = run_case(2, 1, 64, "f16", True, nq, None, seed=8)
    good = out.clone()
    for bad in ([0, 100, 300, 230], [0, 100, 150, 10 ** 12], [-7, 100, 150, 230]):
        out.fill_(7.0)
        tg.tg_attend_prompt(q, k, v, ids(bad, np.int64), None, cfg, out, lse)
        torch.cuda.synchronize()
        assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_ROW
        tg.tg_attn_clear_status(cfg)
        if bad[0] == 0:
            assert torch.equal(out[:100], good[:100])
        else:
            assert torch.equal(out[100:], good[100:]) and (out[:100] == 7.0).all()


def test_prompt_offsets_at_the_ends_of_64_bits():
    # an end so far below its beginning that their difference wraps to a positive number
    import torch
    import logits_processing_token_gb300 as tg
    nq, least = [100, 50, 80], -2 ** 63
    cfg, q, k, v, qo, ko, out, lse = run_case(2, 1, 64, "f16", True, nq, None, seed=9)
    good = out.clone()
    for qb, kb in (([0, 100, least, 230], None), ([0, 100, 150, 230], [0, 100, least, 230]), ([5, least, 150, 230], None),
                   ([0, 100, 2 ** 63 - 1, 230], None)):
        out.fill_(7.0)
        tg.tg_attend_prompt(q, k, v, ids(qb, np.int64), None if kb is None else ids(kb, np.int64), cfg, out, lse)
        torch.cuda.synchronize()
        assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_ROW
        tg.tg_attn_clear_status(cfg)
        if qb[0] == 0:
            assert torch.equal(out[:100], good[:100]) and (out[100:] == 7.0).all()
        else:
            assert torch.equal(out[150:], good[150:]) and (out[:150] == 7.0).all()


@pytest.mark.parametrize("H, G, D, typ, causal", [(2, 1, 128, "bf16", True), (4, 2, 64, "f16", True), (3, 3, 80, "bf16", False)])
def test_prompt_bits_do_not_depend_on_the_neighbours(H, G, D, typ, causal):
    # the rows behind a sequence's end in its last tile are the next one's queries
    import torch
    import logits_processing_token_gb300 as tg
    nq = [700, 41, 333, 20, 505]
    q, k, v, qo, ko = make(H, G, D, typ, nq, nq, 11)
    at = np.concatenate([[0], np.cumsum(nq)])
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ)
    out, lse = torch.empty_like(q.contiguous()), torch.empty(q.shape[:2], device="cuda")
    tg.tg_attend_prompt(q, k, v, qo, None, cfg, out, lse, causal=causal)
    for other in (30.0, float("nan"), 0.0):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for s in (1, 3):
            for t in (q2, k2, v2):
                t[at[s]:at[s + 1]] *= other
        o2, z2 = torch.empty_like(out), torch.empty_like(lse)
        tg.tg_attend_prompt(q2, k2, v2, qo, None, cfg, o2, z2, causal=causal)
        for s in (0, 2, 4):
            rows = slice(int(at[s]), int(at[s + 1]))
            assert torch.equal(o2[rows], out[rows]) and torch.equal(z2[rows], lse[rows]), (other, s)
