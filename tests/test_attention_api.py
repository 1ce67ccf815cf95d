"""The attention calls without a GPU: what they refuse, the structures' layout,
and the oracle's own pins."""
import ctypes
import os
import subprocess
import types

import numpy as np
import pytest

import logits_processing_token_gb300 as tg
from logits_processing_token_gb300 import _build
from oracle import attention_oracle as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tg.load_library()


@pytest.mark.parametrize("struct", [tg.tg_attn_params, tg.tg_cache])
def test_struct_layout_matches_c(struct, tmp_path):
    fields = [f for f, _ in struct._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"tg.h\"\nint main(void){\n"
    src += 'printf("%%zu\\n", sizeof(%s));\n' % struct.__name__
    for f in fields:
        src += 'printf("%%zu\\n", offsetof(%s, %s));\n' % (struct.__name__, f)
    c, exe = str(tmp_path / "t.c"), str(tmp_path / "t")
    open(c, "w").write(src + "return 0;}\n")
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
    vals = [int(x) for x in subprocess.check_output([exe]).split()]
    assert vals[0] == ctypes.sizeof(struct)
    for f, off in zip(fields, vals[1:]):
        assert getattr(struct, f).offset == off, f


GOOD = dict(num_heads=8, num_kv_heads=2, head_dim=64)


@pytest.mark.parametrize("change, unsupported", [
    (dict(num_heads=7), False), (dict(num_heads=0), False), (dict(num_kv_heads=0), False), (dict(num_heads=2048), False),
    (dict(head_dim=0), False), (dict(head_dim=72), True), (dict(head_dim=144), True),
    (dict(dtype=0), False), (dict(dtype="e4m3"), False), (dict(cache_dtype="f16"), False),
    (dict(page_size=0), False), (dict(page_size=24), True), (dict(page_size=2048), False), (dict(page_layout=2), False),
    (dict(scale=-1.0), False), (dict(scale=float("nan")), False), (dict(scale=float("inf")), False),
    (dict(rotary_dim=80, inv_freq=[0.1] * 40), False), (dict(rotary_dim=12, inv_freq=[0.1] * 6), True),
    (dict(rotary_dim=32), False), (dict(rotary_dim=32, inv_freq=[float("inf")] * 16), False),
    (dict(rotary_dim=-16), False), (dict(max_step_tokens=33), False), (dict(max_step_tokens=-1), False),
    (dict(k_scales=[1.0, 1.0]), False), (dict(cache_dtype="e4m3", k_scales=[1.0, 0.0]), False),
    (dict(cache_dtype="e4m3", v_scales=[1.0, float("nan")]), False),
])
def test_create_refuses(lib, change, unsupported):
    p, keep = tg.make_attn_params(**{**GOOD, **change})
    h = ctypes.c_void_p()
    want = tg.TG_ERR_UNSUPPORTED if unsupported else tg.TG_ERR_INVALID_ARGUMENT
    assert lib.tg_attn_create(ctypes.byref(p), ctypes.byref(h), None) == want
    assert not h.value


def test_null_arguments_refused(lib):
    bad = tg.TG_ERR_INVALID_ARGUMENT
    h = ctypes.c_void_p()
    assert lib.tg_attn_create(None, ctypes.byref(h), None) == bad
    assert lib.tg_attn_create(ctypes.byref(tg.make_attn_params(**GOOD)[0]), None, None) == bad
    assert lib.tg_attn_destroy(None) == bad
    assert lib.tg_attn_status_word(None, None) == bad and lib.tg_attn_clear_status(None) == bad
    c = tg.tg_cache()
    assert lib.tg_cache_append(None, 0, None, 0, None, 0, None, 1, ctypes.byref(c), None, None, None, None) == bad
    assert lib.tg_attend_step(None, 0, 1, ctypes.byref(c), None, None, None, None) == bad
    assert lib.tg_attend_prompt(None, 0, None, 0, None, 0, None, None, 1, 1, 1, 1, None, None, None, None) == bad


class _FakeCuda:
    """A CPU tensor that says it is on the GPU: the binding's checks run before any pointer is used."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)


def _fake_cfg():
    import torch
    return types.SimpleNamespace(handle=None, num_heads=4, num_kv_heads=2, head_dim=64, page_size=16, dtype=torch.bfloat16,
                                 cache_dtype=torch.bfloat16, page_shape=(16, 2, 64), max_step_tokens=17)


def test_binding_refuses_wrong_tensors():
    import torch
    cfg, F = _fake_cfg(), _FakeCuda
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    q, kv = F(torch.zeros(5, 4, 64, dtype=bf)), F(torch.zeros(5, 2, 64, dtype=bf))
    pages, table, lens = F(torch.zeros(3, 16, 2, 64, dtype=bf)), F(torch.zeros(2, 2, dtype=i32)), F(torch.zeros(2, dtype=i32))
    off = F(torch.zeros(3, dtype=i64))

    def append(q=q, k=kv, v=kv, off=off, lens=lens, table=table, kp=pages, vp=pages, qo=q, ko=None):
        tg.tg_cache_append(q, k, v, off, lens, table, kp, vp, cfg, qo, ko)

    for what, kw in (("CUDA", dict(k=torch.zeros(5, 2, 64, dtype=bf))),
                     ("dtype", dict(k=F(torch.zeros(5, 2, 64)))),
                     ("must end in", dict(k=F(torch.zeros(5, 3, 64, dtype=bf)))),
                     ("contiguous", dict(k=F(torch.zeros(5, 64, 2, dtype=bf).transpose(1, 2)))),
                     ("same number of tokens", dict(v=F(torch.zeros(4, 2, 64, dtype=bf)))),
                     ("go together", dict(qo=None)),
                     ("k_pages", dict(kp=F(torch.zeros(3, 2, 16, 64, dtype=bf)))),
                     ("v_pages", dict(vp=F(torch.zeros(3, 16, 2, 64)))),
                     ("same number of pages", dict(vp=F(torch.zeros(4, 16, 2, 64, dtype=bf)))),
                     ("page must be contiguous", dict(kp=F(torch.zeros(3, 2, 16, 64, dtype=bf).transpose(1, 2)))),
                     ("page_table", dict(table=F(torch.zeros(2, 2, dtype=i64)))),
                     ("page_table", dict(table=F(torch.zeros(2, 3, dtype=i32).T))),
                     ("kv_lens", dict(lens=F(torch.zeros(1, dtype=i32)))),
                     ("q_offsets", dict(off=F(torch.zeros(2, dtype=i64)))),
                     ("k_out", dict(ko=F(torch.zeros(4, 2, 64, dtype=bf)))),
                     ("q_out", dict(qo=F(torch.zeros(5, 4, 64))))):
        with pytest.raises(ValueError, match=what):
            append(**kw)
    q4 = F(torch.zeros(2, 1, 4, 64, dtype=bf))
    with pytest.raises(ValueError, match="batch, n"):
        tg.tg_attend_step(q, lens, table, pages, pages, cfg, q)
    with pytest.raises(ValueError, match="sequences"):
        tg.tg_attend_step(F(torch.zeros(3, 1, 4, 64, dtype=bf)), lens, table, pages, pages, cfg, q4)
    with pytest.raises(ValueError, match="evenly"):
        tg.tg_attend_step(F(torch.zeros(2, 5, 4, 64, dtype=bf)[:, :3]), lens, table, pages, pages, cfg, q4)
    with pytest.raises(ValueError, match="out holds"):
        tg.tg_attend_step(q4, lens, table, pages, pages, cfg, F(torch.zeros(1, 1, 4, 64, dtype=bf)))
    with pytest.raises(ValueError, match="out_lse"):
        tg.tg_attend_step(q4, lens, table, pages, pages, cfg, q4, F(torch.zeros(2, 1, 3)))
    with pytest.raises(ValueError, match="same number of tokens"):
        tg.tg_attend_prompt(q, kv, F(torch.zeros(4, 2, 64, dtype=bf)), off, None, cfg, q)
    with pytest.raises(ValueError, match="kv_offsets"):
        tg.tg_attend_prompt(q, kv, kv, off, F(torch.zeros(2, dtype=i64)), cfg, q)
    with pytest.raises(ValueError, match="inv_freq"):
        tg.make_attn_params(8, 2, 64, rotary_dim=64, inv_freq=[0.1] * 31)


def test_oracle_attention_pins():
    rng = np.random.default_rng(0)
    k, v = rng.normal(size=(7, 4)), rng.normal(size=(7, 3))
    # one key: its value; equal scores: the mean; no key: 0 and -inf
    out, tol, lse, _ = A.attend(np.stack([rng.normal(size=4), np.zeros(4), np.ones(4)]), k, v, [1, 5, 0], 0.5, "bf16")
    assert np.allclose(out[0], v[0]) and np.allclose(out[1], v[:5].mean(0)) and (out[2] == 0).all()
    assert np.isclose(lse[1], np.log(5)) and np.isneginf(lse[2]) and (tol[:2] > 0).all()
    # weights 3 : 1
    out, _, lse, _ = A.attend([[np.log(3.0), 0.0]], np.eye(2), [[4.0], [8.0]], [2], 1.0, "f16")
    assert np.allclose(out, [[5.0]]) and np.allclose(lse, np.log(4.0))


def test_oracle_rotation_pins():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    # a quarter turn sends (a, b) to (-b, a); the part behind rotary_dim stays
    y, _ = A.rotate(x, [1], [np.pi / 2, 0.0], False)
    assert np.allclose(y[0, 0], [-3, 2, 1, 4, 5, 6, 7, 8])
    y, _ = A.rotate(x, [1], [np.pi / 2, 0.0], True)
    assert np.allclose(y[0, 0], [-2, 1, 3, 4, 5, 6, 7, 8])
    # products of rotated pairs depend on the distance of their positions alone
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 1, 1, 8))
    f = [1.0, 0.3, 0.01, 0.002]
    dots = [float((A.rotate(q, [p + 5], f, False)[0] * A.rotate(k, [p], f, False)[0]).sum()) for p in (0, 17, 400)]
    assert np.allclose(dots, dots[0])


def test_native_marshalling_leaves_refusals_to_the_checks():
    # on tensors that are not on a GPU, or not tensors, the native module makes no call
    import torch
    from logits_processing_token_gb300 import tg as T
    m = T._load_binding()
    h = m.make(0, 4, 2, 64, 16, 2, tg.TG_DTYPE_BF16, tg.TG_DTYPE_BF16, 0, 0, 0)
    bf = torch.bfloat16
    q, kv, pages = torch.zeros(2, 1, 4, 64, dtype=bf), torch.zeros(2, 2, 64, dtype=bf), torch.zeros(3, 16, 2, 64, dtype=bf)
    table, lens, off = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    assert m.step(q, lens, table, pages, pages, h, q, None, None) is None
    assert m.append(None, kv, kv, off, lens, table, pages, pages, h, None, None, None) is None
    assert m.prompt(q[0], kv, kv, off, None, h, q[0], None, True, None) is None
    assert m.step(1, 2, 3, 4, 5, h, 6, 7, 8) is None
    assert m.step(q, lens, table, pages, pages, "no handle", q, None, None) is None
    assert m.step(q) is None


def test_binding_refuses_broadcast_rows():
    # a stride of 0 between rows: one row in memory, however many the shape says
    import torch
    cfg, F = _fake_cfg(), _FakeCuda
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s: torch.zeros(*s, dtype=bf)  # noqa: E731
    pages, table, lens = F(z(3, 16, 2, 64)), F(torch.zeros(3, 2, dtype=i32)), F(torch.zeros(3, dtype=i32))
    off = F(torch.zeros(4, dtype=torch.int64))
    q, kv = z(5, 4, 64), z(5, 2, 64)
    good = dict(q=q, k=kv, v=kv)
    for name, x in (("q", z(1, 4, 64).expand(5, 4, 64)), ("k", z(1, 2, 64).expand(5, 2, 64)), ("v", z(1, 2, 64).expand(5, 2, 64))):
        t = {n: F(x if n == name else y) for n, y in good.items()}
        with pytest.raises(ValueError, match="%s: its rows are one broadcast row" % name):
            tg.tg_cache_append(t["q"], t["k"], t["v"], off, lens, table, pages, pages, cfg, F(q))
        with pytest.raises(ValueError, match="%s: its rows are one broadcast row" % name):
            tg.tg_attend_prompt(t["q"], t["k"], t["v"], off, None, cfg, F(q))
    for x in (z(3, 1, 4, 64).expand(3, 17, 4, 64), z(1, 1, 4, 64).expand(3, 1, 4, 64), z(1, 1, 4, 64).expand(3, 5, 4, 64)):
        with pytest.raises(ValueError, match="q: its rows are one broadcast row"):
            tg.tg_attend_step(F(x), lens, table, pages, pages, cfg, F(z(*x.shape)))
    # the rows of a sequence broadcast over the batch have two spacings
    with pytest.raises(ValueError, match="evenly"):
        tg.tg_attend_step(F(z(1, 5, 4, 64).expand(3, 5, 4, 64)), lens, table, pages, pages, cfg, F(z(3, 5, 4, 64)))
    # one row alone has no spacing, whatever its strides say
    rows = lambda x, heads: tg.tg._head_rows(F(x), "x", heads, cfg)[1]  # noqa: E731
    with pytest.raises(ValueError, match="x: its rows are one broadcast row"):
        rows(z(1, 1, 4, 64).expand(1, 5, 4, 64), 4)
    assert rows(z(1, 4, 64).as_strided((1, 4, 64), (0, 64, 1)), 4) == 256
    assert rows(z(1, 1, 4, 64).as_strided((1, 1, 4, 64), (0, 0, 64, 1)), 4) == 256
    assert rows(z(0, 5, 4, 64), 4) == 256 and rows(z(3, 5, 4, 64), 4) == 256
    assert rows(z(6, 6, 64)[::2, :4], 4) == 768 and rows(z(3, 1, 6, 64)[:, :, :4], 4) == 384
