"""The i8 cache, tg_cache_read and tg_attend_shared without a GPU: what is refused, and
the definition of the codes."""
import ctypes
import types

import numpy as np
import pytest

import logits_processing_token_gb300 as tg
from logits_processing_token_gb300 import _build
from tests.quant_util import quantised
from tests.test_attention_api import GOOD, _FakeCuda

I8 = dict(GOOD, cache_dtype="i8")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tg.load_library()


@pytest.mark.parametrize("change", [dict(k_scales=[1.0, 1.0]), dict(v_scales=[1.0, 1.0]), dict(dtype=tg.TG_DTYPE_I8),
                                    dict(max_shared_tokens=-1), dict(cache_dtype=5)])
def test_create_refuses(lib, change):
    p, keep = tg.make_attn_params(**{**I8, **change})
    h = ctypes.c_void_p()
    assert lib.tg_attn_create(ctypes.byref(p), ctypes.byref(h), None) == tg.TG_ERR_INVALID_ARGUMENT
    assert not h.value


def test_null_arguments_refused(lib):
    bad, c = tg.TG_ERR_INVALID_ARGUMENT, tg.tg_cache()
    assert lib.tg_cache_read(None, 1, ctypes.byref(c), None, None, 0, None, 0, None) == bad
    assert lib.tg_cache_read(None, -1, None, None, None, 0, None, 0, None) == bad
    assert lib.tg_attend_shared(None, 0, 1, ctypes.byref(c), None, None, 0, None, None, None, None) == bad
    assert lib.tg_attend_shared(None, 0, 1, None, None, None, 0, None, None, None, None) == bad


def _cfg(i8=True):
    import torch
    return types.SimpleNamespace(handle=None, num_heads=4, num_kv_heads=2, head_dim=64, page_size=16, dtype=torch.bfloat16,
                                 cache_dtype=torch.uint8 if i8 else torch.bfloat16, max_step_tokens=17, max_shared_tokens=8,
                                 page_shape=(16 * 2 * 68,) if i8 else (16, 2, 64))


def _tensors(i8=True):
    import torch
    F, bf, i32, i64 = _FakeCuda, torch.bfloat16, torch.int32, torch.int64
    size = 16 * 2 * 68
    pages = F(torch.zeros(3, size, dtype=torch.uint8)) if i8 else F(torch.zeros(3, 16, 2, 64, dtype=bf))
    return types.SimpleNamespace(F=F, q=F(torch.zeros(2, 3, 4, 64, dtype=bf)), kv=F(torch.zeros(5, 2, 64, dtype=bf)), pages=pages,
                                 table=F(torch.zeros(2, 2, dtype=i32)), lens=F(torch.zeros(2, dtype=i32)),
                                 off=F(torch.zeros(3, dtype=i64)), prefix=F(torch.zeros(2, dtype=i32)),
                                 lse=F(torch.zeros(2, 3, 4)), size=size)


def test_binding_refuses_wrong_read_tensors():
    import torch
    t, cfg = _tensors(), _cfg()
    bf = torch.bfloat16

    def read(off=t.off, lens=t.lens, table=t.table, kp=t.pages, vp=t.pages, k=t.kv, v=t.kv):
        tg.tg_cache_read(off, lens, table, kp, vp, cfg, k, v)

    for what, kw in (("k or v", dict(k=None, v=None)),
                     ("same number of tokens", dict(v=t.F(torch.zeros(4, 2, 64, dtype=bf)))),
                     ("dtype", dict(k=t.F(torch.zeros(5, 2, 64)))),
                     ("must be \\[tokens", dict(k=t.F(torch.zeros(5, 128, dtype=bf)))),
                     ("must end in", dict(v=t.F(torch.zeros(5, 2, 32, dtype=bf)))),
                     ("broadcast", dict(k=t.F(torch.zeros(1, 2, 64, dtype=bf).expand(5, 2, 64)))),
                     ("contiguous", dict(k=t.F(torch.zeros(5, 64, 2, dtype=bf).transpose(1, 2)))),
                     ("bytes or more", dict(kp=t.F(torch.zeros(3, t.size - 1, dtype=torch.uint8)))),
                     ("bytes or more", dict(vp=t.F(torch.zeros(3, 16, 2, 64, dtype=torch.uint8)))),
                     ("dtype", dict(kp=t.F(torch.zeros(3, t.size, dtype=torch.int8)))),
                     ("page must be contiguous", dict(kp=t.F(torch.zeros(3, 2 * t.size, dtype=torch.uint8)[:, ::2]))),
                     ("same number of pages", dict(vp=t.F(torch.zeros(4, t.size, dtype=torch.uint8)))),
                     ("page_table", dict(table=t.F(torch.zeros(2, 2)))),
                     ("kv_lens", dict(lens=t.F(torch.zeros(1, dtype=torch.int32)))),
                     ("offsets", dict(off=t.F(torch.zeros(2, dtype=torch.int64)))),
                     ("offsets", dict(off=t.F(torch.zeros(3, dtype=torch.int32))))):
        with pytest.raises(ValueError, match=what):
            read(**kw)


@pytest.mark.parametrize("i8", [True, False])
def test_binding_refuses_wrong_shared_tensors(i8):
    import torch
    t, cfg = _tensors(i8), _cfg(i8)
    bf = torch.bfloat16

    def shared(q=t.q, lens=t.lens, table=t.table, kp=t.pages, vp=t.pages, off=t.off, prefix=t.prefix, out=t.q, lse=t.lse):
        tg.tg_attend_shared(q, lens, table, kp, vp, off, prefix, cfg, out, lse)

    for what, kw in (("batch, n", dict(q=t.kv)),
                     ("max_shared_tokens", dict(q=t.F(torch.zeros(3, 3, 4, 64, dtype=bf)))),
                     ("sequences", dict(q=t.F(torch.zeros(1, 3, 4, 64, dtype=bf)))),
                     ("must end in", dict(q=t.F(torch.zeros(2, 3, 2, 64, dtype=bf)))),
                     ("evenly spaced", dict(q=t.F(torch.zeros(2, 4, 4, 64, dtype=bf)[:, :3]))),
                     ("group_offsets", dict(off=t.F(torch.zeros(2, dtype=torch.int64)))),
                     ("group_offsets", dict(off=t.F(torch.zeros(3, dtype=torch.int32)))),
                     ("prefix_lens", dict(prefix=t.F(torch.zeros(2, dtype=torch.int64)))),
                     ("prefix_lens", dict(prefix=torch.zeros(2, dtype=torch.int32))),
                     ("out ", dict(out=t.F(torch.zeros(2, 2, 4, 64, dtype=bf)))),
                     ("out_lse", dict(lse=t.F(torch.zeros(2, 2, 4))))):
        with pytest.raises(ValueError, match=what):
            shared(**kw)


def test_codes_by_hand():
    # 127 steps to the largest magnitude; ties to even; zeros
    x = np.array([[127.0, -127.0, 0.5, 1.5, -2.5, 63.49, 0.0, -0.0], [0.0] * 8, [-2.0, 1.0, 0.0, 2.0, 1.99, 0.0, 0.0, 0.0]])
    q, s = quantised(x)
    assert s[0] == 1.0 and s[1] == 0.0 and s[2] == np.float32(2.0) / np.float32(127.0)
    assert q[0].tolist() == [255, 1, 128, 130, 126, 191, 128, 128] and (q[1] == 128).all()
    assert q[2].tolist() == [1, 192, 128, 255, 254, 128, 128, 128]  # 1 / s = 63.5, to even
