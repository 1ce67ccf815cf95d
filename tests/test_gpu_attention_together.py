"""The quantised cache, its reading back and shared prefixes as they are used together: a prompt
in two chunks, beams of it, and a verify step, over one i8 cache, next to the same over
the values that the cache holds."""
import numpy as np
import pytest

from oracle import attention_oracle as A
from tests.attention_util import check_attention, f64, ids

pytestmark = pytest.mark.gpu

H, G, D, P = 8, 2, 64, 16


@pytest.mark.parametrize("layout, typ", [("token", "bf16"), ("head", "f16")])
def test_chunks_beams_and_verify_over_one_cache(layout, typ):
    import torch
    import logits_processing_token_gb300 as tg
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[typ]
    g = torch.Generator("cuda").manual_seed(0)
    inv = (10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)
    beams, chunks, n = 4, [70, 45], 3
    prompt = sum(chunks)
    cfg = tg.AttnConfig(num_heads=H, num_kv_heads=G, head_dim=D, dtype=typ, cache_dtype="i8", page_size=P, page_layout=layout,
                        rotary_dim=D, inv_freq=inv.tolist(), max_step_tokens=8, max_shared_tokens=beams * 8)
    k_pages, v_pages = (torch.zeros(40, cfg.page_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    random = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(t)  # noqa: E731

    # the prompt, on pages 0 .. of one sequence
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    done = 0
    for m in chunks:
        done += m
        q, k, v = random(m, H, D), random(m, G, D), random(m, G, D)
        lens, off = ids([done], np.int32), ids([0, m], np.int64)
        q2 = torch.empty_like(q)
        tg.tg_cache_append(q, k, v, off, lens, table, k_pages, v_pages, cfg, q2)
        kk, vv = (torch.empty(done, G, D, dtype=t, device="cuda") for _ in range(2))
        all_off = ids([0, done], np.int64)
        tg.tg_cache_read(all_off, lens, table, k_pages, v_pages, cfg, kk, vv)
        out = torch.empty_like(q)
        tg.tg_attend_prompt(q2, kk, vv, off, all_off, cfg, out)
        for h in range(H):
            o, tol, _, _ = A.attend(f64(q2)[:, h], f64(kk)[:, h // 4], f64(vv)[:, h // 4], done - m + 1 + np.arange(m), D ** -0.5, typ)
            assert (np.abs(f64(out)[:, h] - o) <= tol).all()

    # beams: the prompt's whole pages are shared, the page in which it ends is copied
    whole = prompt // P
    rows = torch.full((beams, 10), -1, dtype=torch.int32, device="cuda")
    rows[:, :whole] = table[:, :whole]
    for b in range(beams):
        rows[b, whole:whole + 2] = torch.tensor([8 + 2 * b, 9 + 2 * b])
        for pages in (k_pages, v_pages):
            pages[8 + 2 * b] = pages[int(table[0, whole])]
    groups, prefix = ids([0, beams], np.int64), ids([prompt], np.int32)
    length = prompt
    for m in (1, 1, n):  # two single tokens, then a verify step
        length += m
        lens = ids([length] * beams, np.int32)
        q, k, v = random(beams * m, H, D), random(beams * m, G, D), random(beams * m, G, D)
        q2 = torch.empty_like(q)
        tg.tg_cache_append(q, k, v, ids(np.arange(beams + 1) * m, np.int64), lens, rows, k_pages, v_pages, cfg, q2)
        all_off = ids(np.arange(beams + 1) * length, np.int64)
        kk, vv = (torch.empty(beams * length, G, D, dtype=t, device="cuda") for _ in range(2))
        tg.tg_cache_read(all_off, lens, rows, k_pages, v_pages, cfg, kk, vv)
        for b in range(1, beams):
            assert torch.equal(kk[b * length:b * length + prompt], kk[:prompt])
        q2 = q2.view(beams, m, H, D)
        want = [np.zeros((beams, m, H, D)), np.zeros((beams, m, H, D)), np.zeros((beams, m, H)), np.zeros((beams, m, H))]
        wide = torch.full((beams, -(-(120 << 20) // (2 * G * D * P * beams))), -1, dtype=torch.int32, device="cuda")
        wide[:, :10] = rows
        for b in range(beams):
            for h in range(H):
                # (the 16-bit values that come back are rounded once: half a step of each in keys and values)
                r = A.attend(f64(q2)[b, :, h], f64(kk)[b * length:(b + 1) * length, h // 4], f64(vv)[b * length:(b + 1) * length, h // 4],
                             length - m + 1 + np.arange(m), D ** -0.5, typ, "f16")
                for dst, x in zip(want, r):
                    dst[b, :, h] = x
        half = A.HALF[typ]
        size = np.abs(f64(q2)).sum(-1) * np.abs(f64(kk)).max() * D ** -0.5 * half  # of a score
        want[1] += (2 * size[..., None] + half) * np.abs(f64(vv)).max()
        want[3] += size
        for page_rows in (rows, wide):  # too little to share, and shared
            out, lse = torch.empty_like(q2), torch.empty(beams, m, H, device="cuda")
            tg.tg_attend_shared(q2, lens, page_rows, k_pages, v_pages, groups, prefix, cfg, out, lse)
            check_attention((out, lse), want)
        o2, z2 = torch.empty_like(q2), torch.empty(beams, m, H, device="cuda")
        tg.tg_attend_step(q2, lens, rows, k_pages, v_pages, cfg, o2, z2)
        check_attention((o2, z2), want)
    assert tg.tg_attn_status_word(cfg) == 0
