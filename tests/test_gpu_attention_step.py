"""tg_attend_step against the 64-bit oracle: lengths of zero and one, pages that
end inside a tile, rows that see no key, every type, layout and head grouping."""
import numpy as np
import pytest

from tests.attention_util import Cache, check_attention, f64, ids, step_reference, torch_types

pytestmark = pytest.mark.gpu

CASES = [
    # heads, key heads, dim, type, cache, page, layout, n, lengths
    (4, 1, 128, "bf16", "bf16", 16, "token", 1, [0, 1, 2, 15, 16, 17, 63, 64, 65, 200]),
    (8, 2, 128, "bf16", "bf16", 16, "head", 1, [1000, 3, 0, 129]),
    (16, 2, 64, "f16", "f16", 32, "head", 1, [5, 700, 64]),
    (3, 3, 64, "f16", "f16", 8, "token", 1, [1, 33, 511]),
    (32, 2, 128, "bf16", "e4m3", 64, "head", 1, [300, 0, 1, 77]),
    (8, 4, 64, "f16", "e4m3", 16, "token", 1, [90, 256, 31]),
    (5, 1, 80, "bf16", "bf16", 16, "token", 1, [40, 300]),
    (6, 2, 96, "f16", "f16", 1, "token", 1, [70, 9]),
    (4, 2, 80, "bf16", "e4m3", 1024, "head", 1, [100, 1500]),
    (2, 2, 16, "bf16", "bf16", 2, "head", 1, [65, 4]),
    (7, 1, 112, "f16", "f16", 4, "token", 2, [1, 2, 3, 260]),
    (8, 2, 128, "bf16", "bf16", 16, "token", 5, [0, 1, 4, 5, 6, 64, 67, 333]),
    (8, 2, 128, "bf16", "bf16", 16, "token", 17, [16, 17, 18, 300, 2]),
    (32, 4, 128, "f16", "f16", 128, "head", 17, [20, 200]),
    (8, 1, 64, "f16", "e4m3", 32, "token", 9, [8, 9, 190]),
    (16, 1, 128, "bf16", "e4m3", 32, "token", 32, [31, 100]),
    (4, 4, 64, "bf16", "bf16", 16, "head", 32, [40, 130]),
]


def run_case(H, G, D, typ, cache_kind, page, layout, n, lens, seed=0, with_lse=True, extra=0, shared=False, grow=1.0,
             max_step=32, scale=None):
    import torch
    import logits_processing_token_gb300 as tg
    c = Cache(lens, G, D, cache_kind, page, layout, seed, shared_pool=shared)
    rng = np.random.default_rng(seed + 1)
    q8 = cache_kind == "e4m3"
    ks = rng.uniform(0.02, 0.08, G).astype(np.float32) if q8 else None
    vs = rng.uniform(0.02, 0.08, G).astype(np.float32) if q8 else None
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype=cache_kind, page_size=page,
                        page_layout=layout, k_scales=ks, v_scales=vs, max_step_tokens=max_step, scale=scale)
    B = len(lens)
    t = torch_types()[typ]
    wide = torch.from_numpy(rng.normal(0, 2 * grow, (B, n, H * D + 8 * extra)).astype(np.float32)).cuda().to(t)
    q = wide[..., :H * D].unflatten(2, (H, D))
    out = torch.full((B, n, H, D), float("nan"), device="cuda", dtype=t)
    lse = torch.full((B, n, H), float("nan"), device="cuda") if with_lse else None
    tg.tg_attend_step(q, ids(lens, np.int32), c.device_table(extra), c.k, c.v, cfg, out, lse)
    torch.cuda.synchronize()
    want = step_reference(c, f64(q), n, H // G, scale or 1 / np.sqrt(D), typ, "f16" if q8 else typ, ks, vs)
    check_attention((out, lse), want)
    assert tg.tg_attn_status_word(cfg) == 0
    return cfg, c, q, out, lse


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:8])))
def test_step_matches_oracle(case):
    run_case(*case)


def test_step_strides_and_no_lse():
    # rows of q further apart than they are long, a padded page table, keys and values of a page side by side
    run_case(8, 2, 128, "bf16", "bf16", 16, "token", 3, [50, 0, 129], seed=3, with_lse=False, extra=3, shared=True)
    run_case(4, 2, 64, "f16", "e4m3", 16, "head", 1, [50, 7], seed=4, extra=5, shared=True)


def test_step_long_and_many():
    # one long sequence over the whole GPU, and more sequences than CTAs
    run_case(4, 1, 128, "bf16", "bf16", 64, "token", 1, [40_000], seed=5)
    run_case(2, 1, 64, "f16", "f16", 16, "token", 1, [int(x) for x in np.random.default_rng(6).integers(0, 40, 700)], seed=6)
    run_case(4, 1, 64, "f16", "f16", 16, "token", 20, [3000, 5], seed=7)


def test_step_peaked_weights_and_scale():
    # scores far apart: all the weight on few keys; a scale of the caller's
    run_case(8, 2, 128, "bf16", "bf16", 16, "token", 1, [500, 70], seed=8, grow=20.0)
    run_case(8, 2, 64, "bf16", "e4m3", 16, "token", 4, [500, 70], seed=9, grow=1e-3, scale=3.0)
    run_case(4, 2, 64, "bf16", "e4m3", 16, "token", 1, [90], seed=10, grow=1e4, scale=1e-5)


def test_step_equal_bits_and_stream():
    import torch
    import logits_processing_token_gb300 as tg
    lens = [2000, 0, 17, 900, 64]
    cfg, c, q, out, lse = run_case(8, 2, 128, "bf16", "bf16", 16, "token", 2, lens, seed=11)
    table, kl = c.device_table(), ids(lens, np.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o2, z2 = torch.empty_like(out), torch.empty_like(lse)
        with torch.cuda.stream(side):
            tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, o2, z2)
        side.synchronize()
        assert torch.equal(o2, out) and torch.equal(z2, lse)


def test_step_in_a_graph_follows_the_lengths():
    import torch
    import logits_processing_token_gb300 as tg
    lens = [700, 30, 64]
    cfg, c, q, out, lse = run_case(8, 2, 128, "bf16", "bf16", 16, "token", 1, lens, seed=12)
    kl = ids(lens, np.int32)
    table = c.device_table()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, out, lse)
    for now in (lens, [65, 30, 0], [1, 29, 63]):
        kl.copy_(ids(now, np.int32))
        g.replay()
        torch.cuda.synchronize()
        check_attention((out, lse), step_reference(c, f64(q), 1, 4, 1 / np.sqrt(128), "bf16", "bf16", lens=np.array(now)))


def test_step_bad_pages_and_lengths_are_flagged():
    import torch
    import logits_processing_token_gb300 as tg
    lens = [100, 40, 64]
    cfg, c, q, out, lse = run_case(4, 1, 64, "f16", "f16", 16, "token", 1, lens, seed=13)
    table = c.device_table()
    table[0, 2] = 10 ** 6      # keys 32 .. 47 of sequence 0
    table[1, 0] = -5           # keys 0 .. 15 of sequence 1
    kl = ids([100, 40, 10 ** 6], np.int32)  # longer than its row of the table
    tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, out, lse)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_PAGE | tg.TG_FLAG_BAD_ROW
    tg.tg_attn_clear_status(cfg)
    assert tg.tg_attn_status_word(cfg) == 0
    keep = [np.r_[0:32, 48:100], np.r_[16:40], np.r_[0:0]]
    for x in (c.keys, c.values):
        for b in range(3):
            x[b] = x[b][keep[b]]
    check_attention((out, lse), step_reference(c, f64(q), 1, 4, 1 / np.sqrt(64), "f16", "f16",
                                               lens=np.array([len(k) for k in keep])))
    kl = ids([-1, 40, 64], np.int32)
    table = c.device_table()
    tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, out, lse)
    torch.cuda.synchronize()
    assert tg.tg_attn_status_word(cfg) == tg.TG_FLAG_BAD_ROW
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


def test_step_offsets_past_32_bits():
    # a pool of more than 2^31 elements, the sequence's pages at its far end
    import torch
    import logits_processing_token_gb300 as tg
    G, D, P = 8, 128, 64
    pages = (1 << 31) // (G * D * P) + 40
    k = torch.zeros(pages, P, G, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    L = 1000
    use = np.arange(pages - 1, pages - 1 - -(-L // P), -1)
    g = torch.Generator("cuda").manual_seed(1)
    kk, vv = (torch.randn(L, G, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    pos = torch.arange(L, device="cuda")
    pg = ids(use, np.int64)[pos // P]
    k[pg, pos % P], v[pg, pos % P] = kk, vv
    cfg = tg.AttnConfig(num_heads=8, num_kv_heads=G, head_dim=D, page_size=P)
    q = torch.randn(1, 1, 8, D, generator=g, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty(1, 1, 8, device="cuda")
    tg.tg_attend_step(q, ids([L], np.int32), ids(use[None], np.int32), k, v, cfg, out, lse)
    c = Cache([0], G, D, "bf16", P, "token", 0, fill=False)
    c.keys, c.values = [f64(kk)], [f64(vv)]
    check_attention((out, lse), step_reference(c, f64(q), 1, 1, 1 / np.sqrt(D), "bf16", "bf16", lens=np.array([L])))


@pytest.mark.parametrize("rep, n, typ", [(5, 32, "bf16"), (6, 25, "f16")])
def test_wide_step_bits_do_not_depend_on_the_neighbours(rep, n, typ):
    # a row tile holds 128 / rep tokens: the last one's other rows are the next sequence's
    import torch
    import logits_processing_token_gb300 as tg
    G, D, lens = 2, 128, [2000 + 7 * b for b in range(24)]
    c = Cache(lens, G, D, typ, 16, "token", 14)
    cfg = tg.AttnConfig(num_heads=G * rep, num_kv_heads=G, head_dim=D, dtype=typ, max_step_tokens=32)
    q = (2 * torch.randn(len(lens), n, G * rep, D, generator=torch.Generator("cuda").manual_seed(15), device="cuda")).to(torch_types()[typ])
    kl, table = ids(lens, np.int32), c.device_table()

    def call(q):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        tg.tg_attend_step(q, kl, table, c.k, c.v, cfg, out, lse)
        return out, lse

    out, lse = call(q)
    for other in (30.0, float("nan"), 0.0):
        q2 = q.clone()
        q2[1::2] *= other
        o2, z2 = call(q2)
        assert torch.equal(o2[::2], out[::2]) and torch.equal(z2[::2], lse[::2]), other
