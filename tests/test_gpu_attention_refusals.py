"""What the attention calls refuse when the tensors are on the GPU: an error
before anything is enqueued, and nothing written."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture
def make():
    import torch
    import logits_processing_token_gb300 as tg
    bf, i32 = torch.bfloat16, torch.int32
    cfg = tg.AttnConfig(num_heads=4, num_kv_heads=2, head_dim=64, page_size=16, max_step_tokens=3)
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    return tg, torch, cfg, z, dict(q=z(2, 1, 4, 64), lens=z(2, dtype=i32), table=z(2, 2, dtype=i32), kp=z(3, 16, 2, 64),
                                   vp=z(3, 16, 2, 64), out=z(2, 1, 4, 64) + 7)


def test_step_refusals(make):
    tg, torch, cfg, z, a = make

    def call(**kw):
        x = {**a, **kw}
        tg.tg_attend_step(x["q"], x["lens"], x["table"], x["kp"], x["vp"], x.get("cfg", cfg), x["out"], x.get("lse"))

    for what, kw in (("CUDA", dict(q=a["q"].cpu())), ("dtype", dict(q=a["q"].half())), ("must end in", dict(q=z(2, 1, 2, 64))),
                     ("evenly", dict(q=z(2, 3, 4, 64)[:, :2], out=z(2, 2, 4, 64))),
                     ("contiguous", dict(q=z(2, 1, 4, 128)[..., ::2])), ("v_pages", dict(vp=z(3, 2, 16, 64))),
                     ("same number", dict(vp=z(4, 16, 2, 64))), ("kv_lens", dict(lens=a["lens"].long())),
                     ("page_table", dict(table=a["table"].cpu())), ("out must be contiguous", dict(out=z(4, 1, 4, 64)[::2])),
                     ("out holds", dict(out=z(1, 1, 4, 64))), ("out_lse", dict(lse=z(2, 1, 4))), ("sequences", dict(q=z(3, 1, 4, 64)))):
        with pytest.raises(ValueError, match=what):
            call(**kw)
    # through the C ABI: too many tokens; pointers off 16 bytes; rows that overlap
    for kw in (dict(q=z(2, 4, 4, 64), out=z(2, 4, 4, 64)), dict(q=z(2 * 256 + 1)[1:].view(2, 1, 4, 64)),
               dict(kp=z(3 * 2048 + 1)[1:].view(3, 16, 2, 64)), dict(q=z(300).as_strided((2, 1, 4, 64), (8, 256, 64, 1)))):
        with pytest.raises(tg.TGError, match="INVALID_ARGUMENT"):
            call(**kw)
    torch.cuda.synchronize()
    assert (a["out"] == 7).all() and tg.tg_attn_status_word(cfg) == 0
    call()
    assert (a["out"] == 0).all()
    tg.tg_attend_step(z(0, 1, 4, 64), z(0, dtype=torch.int32), z(0, 2, dtype=torch.int32), a["kp"], a["vp"], cfg, z(0, 1, 4, 64))


def test_prompt_and_append_refusals(make):
    tg, torch, cfg, z, a = make
    q, kv = z(5, 4, 64), z(5, 2, 64)
    off = torch.tensor([0, 2, 5], device="cuda")
    for what, call in (
            ("dtype", lambda: tg.tg_attend_prompt(q, kv.half(), kv, off, None, cfg, q)),
            ("q_offsets", lambda: tg.tg_attend_prompt(q, kv, kv, off.int(), None, cfg, q)),
            ("same number", lambda: tg.tg_attend_prompt(q, kv, kv[:4], off, None, cfg, q)),
            ("out holds", lambda: tg.tg_attend_prompt(q, kv, kv, off, None, cfg, q[:4])),
            ("kv_offsets", lambda: tg.tg_attend_prompt(q, kv, kv, off, off[:2], cfg, q)),
            ("go together", lambda: tg.tg_cache_append(q, kv, kv, off, a["lens"], a["table"], a["kp"], a["vp"], cfg)),
            ("k_out", lambda: tg.tg_cache_append(None, kv, kv, off, a["lens"], a["table"], a["kp"], a["vp"], cfg, None, kv[:3])),
            ("q_offsets", lambda: tg.tg_cache_append(None, kv, kv, off[:2], a["lens"], a["table"], a["kp"], a["vp"], cfg))):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(tg.TGError, match="INVALID_ARGUMENT"):
        tg.tg_attend_prompt(z(5 * 256 + 4)[4:].view(5, 4, 64), kv, kv, off, None, cfg, q)
    # nothing to do is no error
    tg.tg_attend_prompt(z(0, 4, 64), z(0, 2, 64), z(0, 2, 64), torch.zeros(3, dtype=torch.int64, device="cuda"), None, cfg, z(0, 4, 64))
    tg.tg_cache_append(None, z(0, 2, 64), z(0, 2, 64), torch.zeros(3, dtype=torch.int64, device="cuda"), a["lens"], a["table"],
                       a["kp"], a["vp"], cfg)


def test_a_closed_handle_is_refused(make):
    tg, torch, cfg, z, a = make
    cfg.close()
    with pytest.raises(tg.TGError, match="INVALID_ARGUMENT"):
        tg.tg_attend_step(a["q"], a["lens"], a["table"], a["kp"], a["vp"], cfg, a["out"])


def test_broadcast_rows_are_refused(make):
    # one row in memory under a shape of many: nothing is launched
    tg, torch, cfg, z, a = make
    q, kv, off = z(5, 4, 64), z(5, 2, 64), torch.tensor([0, 2, 5], device="cuda")
    out = z(5, 4, 64) + 7
    wide = {"q": z(1, 4, 64).expand(5, 4, 64), "k": z(1, 2, 64).expand(5, 2, 64), "v": z(1, 2, 64).expand(5, 2, 64)}
    for name, x in wide.items():
        t = {"q": q, "k": kv, "v": kv, name: x}
        with pytest.raises(ValueError, match="%s: its rows are one broadcast row" % name):
            tg.tg_attend_prompt(t["q"], t["k"], t["v"], off, None, cfg, out)
        with pytest.raises(ValueError, match="%s: its rows are one broadcast row" % name):
            tg.tg_cache_append(t["q"], t["k"], t["v"], off, a["lens"], a["table"], a["kp"], a["vp"], cfg, out)
    for x in (z(2, 1, 4, 64).expand(2, 3, 4, 64), z(1, 1, 4, 64).expand(2, 1, 4, 64), z(1, 1, 4, 64).expand(2, 3, 4, 64)):
        with pytest.raises(ValueError, match="q: its rows are one broadcast row"):
            tg.tg_attend_step(x, a["lens"], a["table"], a["kp"], a["vp"], cfg, z(2, 3, 4, 64))
    torch.cuda.synchronize()
    assert (out == 7).all() and tg.tg_attn_status_word(cfg) == 0
    # a single row has no spacing
    tg.tg_attend_prompt(z(1, 4, 64).as_strided((1, 4, 64), (0, 64, 1)), kv[:1], kv[:1], torch.tensor([0, 1], device="cuda"), None, cfg, out)
    assert (out[0] == 0).all() and (out[1:] == 7).all()
