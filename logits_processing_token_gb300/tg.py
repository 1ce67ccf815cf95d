"""Python binding of libtg (include/tg.h): argument marshalling only.

Every step of the computation runs in the CUDA kernels of libtg.so.  This
module turns torch CUDA tensors into device pointers, passes the current
stream, and raises :class:`TGError` on a non-zero status.  It never computes
a result itself; if the library is missing it raises instead of falling back.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_char_p, c_float, c_int, c_int32, c_int64, c_uint32, c_uint64, c_void_p

from . import _build

TG_OK = 0
TG_ERR_INVALID_ARGUMENT = -1
TG_ERR_UNSUPPORTED = -2
TG_ERR_CUDA = -3
TG_ERR_OUT_OF_MEMORY = -4

TG_DTYPE_F32, TG_DTYPE_BF16, TG_DTYPE_F16, TG_DTYPE_E4M3, TG_DTYPE_I8 = 0, 1, 2, 3, 4
TG_GREEDY, TG_SAMPLE = 0, 1

TG_FLAG_HISTORY_ID_OUT_OF_RANGE = 0x1
TG_FLAG_BAD_ROW = 0x2
TG_FLAG_SLOW_PATH = 0x4
TG_FLAG_TIMEOUT = 0x8
TG_FLAG_BAD_STATE = 0x10
TG_FLAG_BAD_PAGE = 0x20
TG_MAX_VOCAB = 1 << 18
TG_PROC_BIAS, TG_PROC_SET = 0, 1
TG_MAX_PROCESSORS = 8
TG_MAX_STATE_COLS = 4096
TG_MAX_HEAD_DIM = 128
TG_MAX_STEP_TOKENS = 32
TG_PAGES_TOKEN_HEAD, TG_PAGES_HEAD_TOKEN = 0, 1

# Names of every entry point declared in include/tg.h.
EXPORTS = ("tg_params_init", "tg_config_create", "tg_config_destroy", "tg_select", "tg_select_logprobs", "tg_verify",
           "tg_process", "tg_query_status", "tg_clear_status", "tg_next_num_candidates",
           "tg_status_string", "tg_verify_noalloc", "tg_beam_step", "tg_beam_keep",
           "tg_verify_history", "tg_select_state", "tg_process_state", "tg_set_wait_limit", "tg_status_word",
           "tg_config_view", "tg_config_selection",
           "tg_attn_params_init", "tg_attn_create", "tg_attn_destroy", "tg_attn_status_word", "tg_attn_clear_status",
           "tg_cache_append", "tg_cache_read", "tg_attend_step", "tg_attend_shared", "tg_attend_prompt")
TG_NOALLOC_MAX_BATCH = 1024


class TGError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s failed: %s" % (fn, status_string(status)))


class tg_params(ctypes.Structure):
    _fields_ = [
        ("vocab", c_int32),
        ("logits_dtype", c_int),
        ("mode", c_int),
        ("repetition_penalty", c_float),
        ("no_repeat_ngram_size", c_int32),
        ("bad_words_ids", POINTER(c_int32)),
        ("n_bad_words_ids", c_int32),
        ("suppress_tokens", POINTER(c_int32)),
        ("n_suppress_tokens", c_int32),
        ("begin_suppress_tokens", POINTER(c_int32)),
        ("n_begin_suppress_tokens", c_int32),
        ("eos_token_ids", POINTER(c_int32)),
        ("n_eos_token_ids", c_int32),
        ("min_length", c_int32),
        ("min_new_tokens", c_int32),
        ("forced_bos_token_id", c_int32),
        ("forced_eos_token_ids", POINTER(c_int32)),
        ("n_forced_eos_token_ids", c_int32),
        ("max_new_tokens", c_int32),
        ("temperature", c_float),
        ("top_k", c_int32),
        ("top_p", c_float),
        ("max_batch", c_int32),
        ("bad_word_seq_ids", POINTER(c_int32)),
        ("bad_word_seq_offsets", POINTER(c_int32)),
        ("n_bad_word_seqs", c_int32),
        ("renormalize_logits", c_int32),
        ("processor_kinds", POINTER(c_int32)),
        ("processor_sizes", POINTER(c_int32)),
        ("n_processors", c_int32),
    ]


class tg_attn_params(ctypes.Structure):
    _fields_ = [
        ("num_heads", c_int32),
        ("num_kv_heads", c_int32),
        ("head_dim", c_int32),
        ("dtype", c_int),
        ("cache_dtype", c_int),
        ("page_size", c_int32),
        ("page_layout", c_int),
        ("scale", c_float),
        ("rotary_dim", c_int32),
        ("rotary_interleaved", c_int32),
        ("inv_freq", POINTER(c_float)),
        ("k_scales", POINTER(c_float)),
        ("v_scales", POINTER(c_float)),
        ("max_step_tokens", c_int32),
        ("max_shared_tokens", c_int32),
    ]


class tg_cache(ctypes.Structure):
    _fields_ = [
        ("k_pages", c_void_p),
        ("v_pages", c_void_p),
        ("k_page_stride", c_int64),
        ("v_page_stride", c_int64),
        ("num_pages", c_int32),
        ("page_table", c_void_p),
        ("table_stride", c_int64),
        ("max_pages", c_int32),
        ("kv_lens", c_void_p),
        ("batch", c_int32),
    ]


_lib = None
_binding = None


def _load_binding():
    """The native marshalling module, or None where it is not built for this Python and PyTorch."""
    global _binding
    if _binding is None:
        import importlib.util
        import warnings
        if not _build.binding_current():
            warnings.warn("%s is not built for this Python and PyTorch (__graft_entry__.build() does); the attention calls take "
                          "the slower Python checks" % _build.BINDING)
            return None
        spec = importlib.util.spec_from_file_location("tg_binding", _build.BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _binding = module
    return _binding


def library_path() -> str:
    return _build.LIB


def load_library(path: str | None = None):
    """Load libtg.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError("libtg.so is not built (%s); run __graft_entry__.build()" % path)
    lib = ctypes.CDLL(path)
    lib.tg_params_init.argtypes = [POINTER(tg_params), c_int32]
    lib.tg_params_init.restype = None
    lib.tg_config_create.argtypes = [POINTER(tg_params), POINTER(c_void_p), c_void_p]
    lib.tg_status_word.argtypes = [c_void_p, POINTER(c_uint32)]
    lib.tg_status_word.restype = c_int
    lib.tg_config_destroy.argtypes = [c_void_p]
    lib.tg_select.argtypes = [c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                              c_void_p, c_void_p]
    lib.tg_select_logprobs.argtypes = [c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_void_p]
    lib.tg_verify.argtypes = [c_void_p, c_int32, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                              c_void_p, c_void_p]
    lib.tg_verify_history.argtypes = [c_void_p, c_int32, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    lib.tg_verify_history.restype = c_int
    lib.tg_verify_noalloc.argtypes = [c_void_p, c_int32, c_int32, c_void_p, c_int32, POINTER(tg_params), c_void_p,
                                      c_void_p, c_void_p, c_void_p]
    lib.tg_verify_noalloc.restype = c_int
    lib.tg_set_wait_limit.argtypes = [c_uint64]
    lib.tg_set_wait_limit.restype = c_int
    lib.tg_process.argtypes = [c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                               c_void_p, c_void_p, c_void_p]
    lib.tg_select_state.argtypes = [c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    lib.tg_select_state.restype = c_int
    lib.tg_process_state.argtypes = [c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    lib.tg_process_state.restype = c_int
    lib.tg_query_status.argtypes = [c_void_p, POINTER(c_uint32), POINTER(c_uint64)]
    lib.tg_clear_status.argtypes = [c_void_p]
    lib.tg_beam_step.argtypes = [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    lib.tg_beam_step.restype = c_int
    lib.tg_beam_keep.argtypes = [c_void_p, c_int32]
    lib.tg_beam_keep.restype = c_int32
    lib.tg_next_num_candidates.argtypes = [c_int32, c_int32, c_int32]
    lib.tg_next_num_candidates.restype = c_int32
    lib.tg_status_string.argtypes = [c_int]
    lib.tg_status_string.restype = c_char_p
    lib.tg_attn_params_init.argtypes = [POINTER(tg_attn_params), c_int32, c_int32, c_int32]
    lib.tg_attn_params_init.restype = None
    lib.tg_attn_create.argtypes = [POINTER(tg_attn_params), POINTER(c_void_p), c_void_p]
    lib.tg_attn_destroy.argtypes = [c_void_p]
    lib.tg_attn_status_word.argtypes = [c_void_p, POINTER(c_uint32)]
    lib.tg_attn_clear_status.argtypes = [c_void_p]
    lib.tg_cache_append.argtypes = [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int32,
                                    POINTER(tg_cache), c_void_p, c_void_p, c_void_p, c_void_p]
    lib.tg_attend_step.argtypes = [c_void_p, c_int64, c_int32, POINTER(tg_cache), c_void_p, c_void_p, c_void_p, c_void_p]
    lib.tg_cache_read.argtypes = [c_void_p, c_int32, POINTER(tg_cache), c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p]
    lib.tg_attend_shared.argtypes = [c_void_p, c_int64, c_int32, POINTER(tg_cache), c_void_p, c_void_p, c_int32, c_void_p,
                                     c_void_p, c_void_p, c_void_p]
    lib.tg_attend_prompt.argtypes = [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_int32,
                                     c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p]
    for fn in ("tg_attn_create", "tg_attn_destroy", "tg_attn_status_word", "tg_attn_clear_status", "tg_cache_append",
               "tg_cache_read", "tg_attend_step", "tg_attend_shared", "tg_attend_prompt"):
        getattr(lib, fn).restype = c_int
    for fn in ("tg_config_create", "tg_config_destroy", "tg_select", "tg_select_logprobs", "tg_verify", "tg_process",
               "tg_query_status", "tg_clear_status"):
        getattr(lib, fn).restype = c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().tg_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != TG_OK:
        raise TGError(fn, status)


def _ids(seq):
    seq = [int(t) for t in (seq or ())]
    arr = (c_int32 * max(1, len(seq)))(*seq) if seq else None
    return arr, len(seq)


def make_params(vocab: int, logits_dtype="f32", mode="greedy", repetition_penalty=1.0,
                no_repeat_ngram_size=0, bad_words_ids=(), suppress_tokens=(), begin_suppress_tokens=(),
                eos_token_ids=(), min_length=0, min_new_tokens=0, forced_bos_token_id=-1,
                forced_eos_token_ids=(), max_new_tokens=0, temperature=1.0, top_k=0, top_p=1.0,
                max_batch=0, bad_word_seqs=(), renormalize_logits=False, processors=()):
    """A filled tg_params plus the ctypes arrays its pointers refer to."""
    lib = load_library()
    p = tg_params()
    lib.tg_params_init(ctypes.byref(p), int(vocab))
    p.logits_dtype = {"f32": TG_DTYPE_F32, "bf16": TG_DTYPE_BF16}[logits_dtype] if isinstance(logits_dtype, str) else int(logits_dtype)
    p.mode = {"greedy": TG_GREEDY, "sample": TG_SAMPLE}[mode] if isinstance(mode, str) else int(mode)
    p.repetition_penalty = float(repetition_penalty)
    p.no_repeat_ngram_size = int(no_repeat_ngram_size)
    keep = []
    for name, seq in (("bad_words_ids", bad_words_ids), ("suppress_tokens", suppress_tokens),
                      ("begin_suppress_tokens", begin_suppress_tokens), ("eos_token_ids", eos_token_ids),
                      ("forced_eos_token_ids", forced_eos_token_ids)):
        arr, n = _ids(seq)
        keep.append(arr)
        setattr(p, name, ctypes.cast(arr, POINTER(c_int32)) if arr is not None else None)
        setattr(p, "n_" + name, n)
    p.min_length = int(min_length)
    p.min_new_tokens = int(min_new_tokens)
    p.forced_bos_token_id = int(forced_bos_token_id)
    p.max_new_tokens = int(max_new_tokens)
    p.temperature = float(temperature)
    p.top_k = int(top_k)
    p.top_p = float(top_p)
    p.max_batch = int(max_batch)
    p.renormalize_logits = 1 if renormalize_logits else 0
    # bad words of one or more tokens: ids back to back, then n + 1 offsets
    seqs = [list(map(int, s)) for s in bad_word_seqs]
    if seqs:
        flat = [t for s in seqs for t in s]
        offs = [0]
        for s in seqs:
            offs.append(offs[-1] + len(s))
        ids_arr, _ = _ids(flat)
        off_arr, _ = _ids(offs)
        keep += [ids_arr, off_arr]
        p.bad_word_seq_ids = ctypes.cast(ids_arr, POINTER(c_int32))
        p.bad_word_seq_offsets = ctypes.cast(off_arr, POINTER(c_int32))
        p.n_bad_word_seqs = len(seqs)
    # the task's processors: (kind, size) pairs, kind "bias" / "set" or TG_PROC_*
    procs = [(({"bias": TG_PROC_BIAS, "set": TG_PROC_SET}[k] if isinstance(k, str) else int(k)), int(n))
             for k, n in processors]
    if procs:
        kinds_arr, _ = _ids([k for k, _ in procs])
        sizes_arr, _ = _ids([n for _, n in procs])
        keep += [kinds_arr, sizes_arr]
        p.processor_kinds = ctypes.cast(kinds_arr, POINTER(c_int32))
        p.processor_sizes = ctypes.cast(sizes_arr, POINTER(c_int32))
        p.n_processors = len(procs)
    return p, keep


class Config:
    """Owns a tg_config* (tg_config_create / tg_config_destroy)."""

    def __init__(self, stream=None, **params):
        lib = load_library()
        p, keep = make_params(**params)
        h = c_void_p()
        # the uploads go on `stream` (a torch stream), or on the default stream
        st = c_void_p(stream.cuda_stream) if stream is not None else None
        _check("tg_config_create", lib.tg_config_create(ctypes.byref(p), ctypes.byref(h), st))
        self.handle = h
        self.params = dict(params)
        del keep

    def close(self):
        if self.handle:
            load_library().tg_config_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _ptr(t, name, dtypes=None, allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError("%s is required" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    return c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return c_void_p(stream.cuda_stream)


def _logit_dtypes():
    import torch
    return (torch.float32, torch.bfloat16, torch.int16, torch.uint16)


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _check_logits(t, cfg, name):
    """The library reads rows of cfg's element type through a raw pointer:
    the tensor's element size must match it and its last dimension must be V."""
    want = 2 if cfg.params.get("logits_dtype", "f32") in ("bf16", 1) else 4
    _need(t.element_size() == want, "%s has %d-byte elements; the config expects %d-byte logits"
          % (name, t.element_size(), want))
    _need(int(t.shape[-1]) == int(cfg.params["vocab"]), "%s has %d columns; the config's vocab is %d"
          % (name, int(t.shape[-1]), int(cfg.params["vocab"])))


def _check_len(t, n, name):
    if t is not None:
        _need(t.numel() >= n, "%s holds %d elements; the call needs %d" % (name, t.numel(), n))


def tg_select(logits, hist_ids, hist_offsets, prompt_lens, cfg: Config, uniforms, out_ids, stream=None,
              out_logprobs=None):
    """logits [B, V]; hist_offsets [B+1]; prompt_lens [B]; uniforms [B] (sampling); out_ids [B];
    out_logprobs [B] f32 or None (given: tg_select_logprobs, the token's log-probability per row).
    The history ids that hist_offsets point at are not bounds-checked here: they live on the device."""
    import torch
    _need(logits.dim() == 2, "logits must be [B, V]")
    _check_logits(logits, cfg, "logits")
    B, V = int(logits.shape[0]), int(logits.shape[-1])
    _check_len(hist_offsets, B + 1, "hist_offsets")
    _check_len(prompt_lens, B, "prompt_lens")
    _check_len(uniforms, B, "uniforms")
    _check_len(out_ids, B, "out_ids")
    _check_len(out_logprobs, B, "out_logprobs")
    args = [_ptr(logits, "logits", _logit_dtypes()), B, V,
            _ptr(hist_ids, "hist_ids", (torch.int32,), allow_none=True) if hist_ids is not None and hist_ids.numel() else None,
            _ptr(hist_offsets, "hist_offsets", (torch.int64,)), _ptr(prompt_lens, "prompt_lens", (torch.int32,)),
            cfg.handle, _ptr(uniforms, "uniforms", (torch.float32,), allow_none=True),
            _ptr(out_ids, "out_ids", (torch.int32,))]
    lib = load_library()
    if out_logprobs is None:
        st = lib.tg_select(*args, _stream(stream))
        _check("tg_select", st)
    else:
        st = lib.tg_select_logprobs(*args, _ptr(out_logprobs, "out_logprobs", (torch.float32,)), _stream(stream))
        _check("tg_select_logprobs", st)
    return out_ids


def _state_cols(cfg):
    return sum(int(n) for _, n in cfg.params.get("processors", ()))


def tg_select_state(logits, hist_ids, hist_offsets, prompt_lens, cfg: Config, state_ids, state_values, uniforms,
                    out_ids, out_logprobs=None, stream=None):
    """tg_select with the config's task processors: state_ids int32 [B, S] and state_values f32
    [B, S] (S = the processors' columns); out_logprobs [B] f32 or None."""
    import torch
    _need(logits.dim() == 2, "logits must be [B, V]")
    _check_logits(logits, cfg, "logits")
    B, V = int(logits.shape[0]), int(logits.shape[-1])
    S = _state_cols(cfg)
    _check_len(hist_offsets, B + 1, "hist_offsets")
    _check_len(prompt_lens, B, "prompt_lens")
    _check_len(state_ids, B * S, "state_ids")
    _check_len(state_values, B * S, "state_values")
    _check_len(uniforms, B, "uniforms")
    _check_len(out_ids, B, "out_ids")
    _check_len(out_logprobs, B, "out_logprobs")
    st = load_library().tg_select_state(
        _ptr(logits, "logits", _logit_dtypes()), B, V,
        _ptr(hist_ids, "hist_ids", (torch.int32,), allow_none=True) if hist_ids is not None and hist_ids.numel() else None,
        _ptr(hist_offsets, "hist_offsets", (torch.int64,)), _ptr(prompt_lens, "prompt_lens", (torch.int32,)),
        cfg.handle, _ptr(state_ids, "state_ids", (torch.int32,)), _ptr(state_values, "state_values", (torch.float32,)),
        _ptr(uniforms, "uniforms", (torch.float32,), allow_none=True), _ptr(out_ids, "out_ids", (torch.int32,)),
        _ptr(out_logprobs, "out_logprobs", (torch.float32,), allow_none=True), _stream(stream))
    _check("tg_select_state", st)
    return out_ids


def tg_process_state(logits, hist_ids, hist_offsets, prompt_lens, cfg: Config, state_ids, state_values, out_scores,
                     out_banbits=None, out_probs=None, stream=None):
    """tg_process with the config's task processors (state as tg_select_state)."""
    import torch
    _need(logits.dim() == 2, "logits must be [B, V]")
    _check_logits(logits, cfg, "logits")
    B, V = int(logits.shape[0]), int(logits.shape[-1])
    S = _state_cols(cfg)
    _check_len(hist_offsets, B + 1, "hist_offsets")
    _check_len(prompt_lens, B, "prompt_lens")
    _check_len(state_ids, B * S, "state_ids")
    _check_len(state_values, B * S, "state_values")
    _check_len(out_scores, B * V, "out_scores")
    _check_len(out_banbits, B * ((V + 31) // 32), "out_banbits")
    _check_len(out_probs, B * V, "out_probs")
    st = load_library().tg_process_state(
        _ptr(logits, "logits", _logit_dtypes()), B, V,
        _ptr(hist_ids, "hist_ids", (torch.int32,)) if hist_ids is not None and hist_ids.numel() else None,
        _ptr(hist_offsets, "hist_offsets", (torch.int64,)), _ptr(prompt_lens, "prompt_lens", (torch.int32,)),
        cfg.handle, _ptr(state_ids, "state_ids", (torch.int32,)), _ptr(state_values, "state_values", (torch.float32,)),
        _ptr(out_scores, "out_scores", (torch.float32,)),
        _ptr(out_banbits, "out_banbits", (torch.int32, torch.uint32), allow_none=True),
        _ptr(out_probs, "out_probs", (torch.float32,), allow_none=True), _stream(stream))
    _check("tg_process_state", st)


def tg_beam_keep(cfg: Config, num_beams: int) -> int:
    """Candidates a prompt keeps per beam step: max(2, 1 + eos ids) * num_beams."""
    n = load_library().tg_beam_keep(cfg.handle, int(num_beams))
    _need(n > 0, "num_beams must be >= 1")
    return int(n)


def tg_beam_step(logits, beam_scores, hist_ids, hist_offsets, prompt_lens, cfg: Config, num_beams: int,
                 out_scores, out_tokens, out_beams, stream=None):
    """logits [P * num_beams, V]; beam_scores [P * num_beams] f32; hist_offsets [P * num_beams + 1];
    prompt_lens [P * num_beams]; out_scores f32, out_tokens and out_beams int32, each [P, keep]."""
    import torch
    _need(logits.dim() == 2, "logits must be [P * num_beams, V]")
    _check_logits(logits, cfg, "logits")
    R, V = int(logits.shape[0]), int(logits.shape[-1])
    nb = int(num_beams)
    _need(nb >= 1 and R % nb == 0, "the rows must be num_beams per prompt")
    P = R // nb
    keep = tg_beam_keep(cfg, nb)
    _check_len(beam_scores, R, "beam_scores")
    _check_len(hist_offsets, R + 1, "hist_offsets")
    _check_len(prompt_lens, R, "prompt_lens")
    for t, name in ((out_scores, "out_scores"), (out_tokens, "out_tokens"), (out_beams, "out_beams")):
        _check_len(t, P * keep, name)
    st = load_library().tg_beam_step(
        _ptr(logits, "logits", _logit_dtypes()), P, nb, V, _ptr(beam_scores, "beam_scores", (torch.float32,)),
        _ptr(hist_ids, "hist_ids", (torch.int32,), allow_none=True) if hist_ids is not None and hist_ids.numel() else None,
        _ptr(hist_offsets, "hist_offsets", (torch.int64,)), _ptr(prompt_lens, "prompt_lens", (torch.int32,)),
        cfg.handle, _ptr(out_scores, "out_scores", (torch.float32,)), _ptr(out_tokens, "out_tokens", (torch.int32,)),
        _ptr(out_beams, "out_beams", (torch.int32,)), _stream(stream))
    _check("tg_beam_step", st)
    return out_scores, out_tokens, out_beams


def tg_verify(target_logits, cand_ids, K: int, cfg: Config, uniforms, out_match, out_next, stream=None):
    """target_logits [B, K+1, V]; cand_ids [B, K]; uniforms [B, K+1] (sampling);
    out_match [B]; out_next [B, K+1]."""
    import torch
    _need(target_logits.dim() == 3 and int(target_logits.shape[1]) == int(K) + 1,
          "target_logits must be [B, K+1, V]")
    _check_logits(target_logits, cfg, "target_logits")
    B, V = int(target_logits.shape[0]), int(target_logits.shape[-1])
    _check_len(cand_ids, B * int(K), "cand_ids")
    _check_len(uniforms, B * (int(K) + 1), "uniforms")
    _check_len(out_match, B, "out_match")
    _check_len(out_next, B * (int(K) + 1), "out_next")
    st = load_library().tg_verify(
        _ptr(target_logits, "target_logits", _logit_dtypes()), B, V, _ptr(cand_ids, "cand_ids", (torch.int32,)),
        int(K), cfg.handle, _ptr(uniforms, "uniforms", (torch.float32,), allow_none=True),
        _ptr(out_match, "out_match", (torch.int32,)), _ptr(out_next, "out_next", (torch.int32,)), _stream(stream))
    _check("tg_verify", st)
    return out_match, out_next


def tg_verify_history(target_logits, cand_ids, K: int, hist_ids, hist_offsets, prompt_lens, cfg: Config, uniforms,
                      out_match, out_next, stream=None):
    """tg_verify with the processors at every position: position j of row b sees
    the row's history (hist_offsets [B+1], prompt_lens [B]) and its first j candidates."""
    import torch
    _need(target_logits.dim() == 3 and int(target_logits.shape[1]) == int(K) + 1,
          "target_logits must be [B, K+1, V]")
    _check_logits(target_logits, cfg, "target_logits")
    B, V = int(target_logits.shape[0]), int(target_logits.shape[-1])
    _check_len(cand_ids, B * int(K), "cand_ids")
    _check_len(hist_offsets, B + 1, "hist_offsets")
    _check_len(prompt_lens, B, "prompt_lens")
    _check_len(uniforms, B * (int(K) + 1), "uniforms")
    _check_len(out_match, B, "out_match")
    _check_len(out_next, B * (int(K) + 1), "out_next")
    st = load_library().tg_verify_history(
        _ptr(target_logits, "target_logits", _logit_dtypes()), B, V, _ptr(cand_ids, "cand_ids", (torch.int32,)),
        int(K),
        _ptr(hist_ids, "hist_ids", (torch.int32,), allow_none=True) if hist_ids is not None and hist_ids.numel() else None,
        _ptr(hist_offsets, "hist_offsets", (torch.int64,)), _ptr(prompt_lens, "prompt_lens", (torch.int32,)),
        cfg.handle, _ptr(uniforms, "uniforms", (torch.float32,), allow_none=True),
        _ptr(out_match, "out_match", (torch.int32,)), _ptr(out_next, "out_next", (torch.int32,)), _stream(stream))
    _check("tg_verify_history", st)
    return out_match, out_next


def tg_process(logits, hist_ids, hist_offsets, prompt_lens, cfg: Config, out_scores, out_banbits=None,
               out_probs=None, stream=None):
    import torch
    _need(logits.dim() == 2, "logits must be [B, V]")
    _check_logits(logits, cfg, "logits")
    B, V = int(logits.shape[0]), int(logits.shape[-1])
    _check_len(hist_offsets, B + 1, "hist_offsets")
    _check_len(prompt_lens, B, "prompt_lens")
    _check_len(out_scores, B * V, "out_scores")
    _check_len(out_banbits, B * ((V + 31) // 32), "out_banbits")
    _check_len(out_probs, B * V, "out_probs")
    st = load_library().tg_process(
        _ptr(logits, "logits", _logit_dtypes()), B, V,
        _ptr(hist_ids, "hist_ids", (torch.int32,)) if hist_ids is not None and hist_ids.numel() else None,
        _ptr(hist_offsets, "hist_offsets", (torch.int64,)), _ptr(prompt_lens, "prompt_lens", (torch.int32,)),
        cfg.handle, _ptr(out_scores, "out_scores", (torch.float32,)),
        _ptr(out_banbits, "out_banbits", (torch.int32, torch.uint32), allow_none=True),
        _ptr(out_probs, "out_probs", (torch.float32,), allow_none=True), _stream(stream))
    _check("tg_process", st)


def tg_query_status(cfg: Config):
    f, s = c_uint32(), c_uint64()
    _check("tg_query_status", load_library().tg_query_status(cfg.handle, ctypes.byref(f), ctypes.byref(s)))
    return int(f.value), int(s.value)


def tg_status_word(cfg: Config) -> int:
    """The sticky status bits (synchronous)."""
    f = c_uint32()
    _check("tg_status_word", load_library().tg_status_word(cfg.handle, ctypes.byref(f)))
    return int(f.value)


def tg_clear_status(cfg: Config):
    _check("tg_clear_status", load_library().tg_clear_status(cfg.handle))


def tg_set_wait_limit(cycles: int):
    """Testing: the select/verify kernels give up a bulk-copy wait, and the attention kernels
    any wait, after ``cycles`` SM cycles (0 restores the default of about one second)."""
    lib = load_library()
    _check("tg_set_wait_limit", lib.tg_set_wait_limit(int(cycles)))


def tg_next_num_candidates(K: int, n_match: int, K_max: int) -> int:
    return int(load_library().tg_next_num_candidates(int(K), int(n_match), int(K_max)))


def tg_status_string(status: int) -> str:
    return status_string(status)


_ATTN_DTYPES = {"bf16": TG_DTYPE_BF16, "f16": TG_DTYPE_F16, "e4m3": TG_DTYPE_E4M3, "i8": TG_DTYPE_I8}
_PAGE_LAYOUTS = {"token": TG_PAGES_TOKEN_HEAD, "head": TG_PAGES_HEAD_TOKEN}


def make_attn_params(num_heads, num_kv_heads, head_dim, dtype="bf16", cache_dtype=None, page_size=16,
                     page_layout="token", scale=0.0, rotary_dim=0, rotary_interleaved=False, inv_freq=None,
                     k_scales=None, v_scales=None, max_step_tokens=0, max_shared_tokens=0):
    """A filled tg_attn_params plus the ctypes arrays its pointers refer to."""
    p = tg_attn_params()
    load_library().tg_attn_params_init(ctypes.byref(p), int(num_heads), int(num_kv_heads), int(head_dim))
    p.dtype = _ATTN_DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    p.cache_dtype = p.dtype if cache_dtype is None else _ATTN_DTYPES[cache_dtype] if isinstance(cache_dtype, str) else int(cache_dtype)
    p.page_size = int(page_size)
    p.page_layout = _PAGE_LAYOUTS[page_layout] if isinstance(page_layout, str) else int(page_layout)
    p.scale = float(scale or 0.0)
    p.rotary_dim = int(rotary_dim)
    p.rotary_interleaved = 1 if rotary_interleaved else 0
    keep = []
    for name, seq, n in (("inv_freq", inv_freq, p.rotary_dim // 2), ("k_scales", k_scales, p.num_kv_heads),
                         ("v_scales", v_scales, p.num_kv_heads)):
        if seq is None:
            continue
        seq = [float(x) for x in seq]
        if len(seq) != n and not (name == "inv_freq" and n <= 0):
            raise ValueError("%s holds %d values; the settings need %d" % (name, len(seq), n))
        arr = (c_float * max(1, len(seq)))(*seq)
        keep.append(arr)
        setattr(p, name, ctypes.cast(arr, POINTER(c_float)))
    p.max_step_tokens = int(max_step_tokens)
    p.max_shared_tokens = int(max_shared_tokens)
    return p, keep


class AttnConfig:
    """Owns a tg_attn* (tg_attn_create / tg_attn_destroy); keyword arguments as make_attn_params.

    page_shape is the shape of a page; page_bytes what a page takes, up to the next 16 bytes.  An i8 cache's pages are
    rows of page_bytes (or more) of a uint8 tensor: codes, then scales (include/tg.h)."""

    def __init__(self, stream=None, **params):
        import torch
        lib = load_library()
        p, keep = make_attn_params(**params)
        h = c_void_p()
        self.handle = None
        st = c_void_p(stream.cuda_stream) if stream is not None else None
        _check("tg_attn_create", lib.tg_attn_create(ctypes.byref(p), ctypes.byref(h), st))
        self.handle = h
        del keep
        types = {TG_DTYPE_BF16: torch.bfloat16, TG_DTYPE_F16: torch.float16, TG_DTYPE_E4M3: torch.float8_e4m3fn,
                 TG_DTYPE_I8: torch.uint8}
        self.num_heads, self.num_kv_heads, self.head_dim = p.num_heads, p.num_kv_heads, p.head_dim
        self.page_size, self.max_step_tokens = p.page_size, p.max_step_tokens or 17
        self.dtype, self.cache_dtype = types[p.dtype], types[p.cache_dtype]
        G, P, D = p.num_kv_heads, p.page_size, p.head_dim
        self.page_shape = (P, G, D) if p.page_layout == TG_PAGES_TOKEN_HEAD else (G, P, D)
        self.max_shared_tokens = p.max_shared_tokens
        i8 = p.cache_dtype == TG_DTYPE_I8
        self.page_bytes = -(-P * G * (D * self.cache_dtype.itemsize + (4 if i8 else 0)) // 16) * 16
        if i8:
            self.page_shape = (P * G * (D + 4),)
        calls = [ctypes.cast(f, c_void_p).value for f in (lib.tg_cache_append, lib.tg_attend_step, lib.tg_attend_prompt,
                                                          lib.tg_cache_read, lib.tg_attend_shared)]
        native = _load_binding()
        page = (self.page_shape + (0,))[:2]
        self._native = native and native.make(h.value, p.num_heads, G, D, *page, p.dtype, p.cache_dtype, *calls)

    def close(self):
        if self.handle:
            self._native = None
            load_library().tg_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# The attention calls run once or more per layer of a decode step: the native
# module (csrc/tg_binding.cpp) checks and passes on a call whose tensors are as
# they should be.  It returns None for any other, and the checks below then say
# what is wrong with it (or, where the module is not built, pass the call on).

def _head_rows(t, name, heads, cfg):
    """Pointer and row stride of a [.., heads, D] tensor whose heads are
    contiguous and whose rows are evenly spaced."""
    D = cfg.head_dim
    *lead, h, d = t.shape
    *rows, sh, sd = t.stride()
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != cfg.dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, cfg.dtype))
    if h != heads or d != D:
        raise ValueError("%s must end in [%d, %d], not %s" % (name, heads, D, (h, d)))
    if sd != 1 or (sh != D and heads > 1):
        raise ValueError("%s: a row's heads must be contiguous" % name)
    if min(lead) == 0 or max(lead) == 1:
        return t.data_ptr(), heads * D  # no row, or one
    row = rows[-1] if lead[-1] > 1 else rows[0]
    if row == 0:
        raise ValueError("%s: its rows are one broadcast row" % name)
    if len(lead) == 2 and min(lead) > 1 and rows[0] != row * lead[1]:  # [batch, n, heads, D]: one spacing for all rows
        raise ValueError("%s: its rows must be evenly spaced" % name)
    return t.data_ptr(), row


def _whole(t, name, dtype, numel):
    """Pointer of a contiguous tensor of at least numel elements."""
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.numel() < numel:
        raise ValueError("%s holds %d elements; the call needs %d" % (name, t.numel(), numel))
    return t.data_ptr()


def _pages(t, name, cfg):
    """Pointer, page stride and number of pages."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != cfg.cache_dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, cfg.cache_dtype))
    if len(cfg.page_shape) == 1:  # i8: rows of bytes
        if t.dim() != 2 or t.shape[1] < cfg.page_shape[0]:
            raise ValueError("%s must be [pages, %d bytes or more], not %s" % (name, cfg.page_shape[0], tuple(t.shape)))
        if t.stride(1) != 1:
            raise ValueError("%s: a page must be contiguous" % name)
        n, size = t.shape
        return t.data_ptr(), t.stride(0) if n > 1 else -(-size // 16) * 16, n
    n, x, y, D = (*t.shape, 0, 0, 0, 0)[:4]
    if t.dim() != 4 or (x, y, D) != cfg.page_shape:
        raise ValueError("%s must be [pages, %d, %d, %d], not %s" % ((name,) + cfg.page_shape + (tuple(t.shape),)))
    sp, sx, sy, sd = t.stride()
    if sd != 1 or (sy != D and y > 1) or (sx != y * D and x > 1):
        raise ValueError("%s: a page must be contiguous" % name)
    return t.data_ptr(), sp if n > 1 else x * y * D, n


def _cache(cfg, k_pages, v_pages, page_table, kv_lens):
    """The tg_cache of a call."""
    import torch
    kp, ks, pages = _pages(k_pages, "k_pages", cfg)
    vp, vs, vpages = _pages(v_pages, "v_pages", cfg)
    if vpages != pages:
        raise ValueError("k_pages and v_pages must hold the same number of pages")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_cuda:
        raise ValueError("page_table must be a CUDA int32 tensor [batch, max_pages]")
    B, most = page_table.shape
    row, one = page_table.stride()
    if one != 1 and most > 1:
        raise ValueError("page_table: a row must be contiguous")
    return tg_cache(kp, vp, ks, vs, pages, page_table.data_ptr(), row if B > 1 else most, most,
                    _whole(kv_lens, "kv_lens", torch.int32, B), B), B


def tg_cache_append(q, k, v, q_offsets, kv_lens, page_table, k_pages, v_pages, cfg: AttnConfig, q_out=None,
                    k_out=None, stream=None):
    """q [T, H, D] (or None), k and v [T, G, D]: the new tokens of all sequences, rows evenly spaced;
    q_offsets int64 [B + 1]; kv_lens int32 [B], the new tokens included; page_table int32 [B, max_pages];
    k_pages and v_pages [pages, page_size, G, D] or [pages, G, page_size, D] as the config says (i8: uint8 [pages, page_bytes]);
    q_out [T, H, D] and k_out [T, G, D] (or None) take the rotated queries and keys."""
    native = getattr(cfg, "_native", None)
    if native is not None:
        st = _binding.append(q, k, v, q_offsets, kv_lens, page_table, k_pages, v_pages, native, q_out, k_out,
                             None if stream is None else stream.cuda_stream)
        if st is not None:
            return _check("tg_cache_append", st)
    import torch
    H, G, D = cfg.num_heads, cfg.num_kv_heads, cfg.head_dim
    if k.dim() != 3 or v.dim() != 3 or (q is not None and q.dim() != 3):
        raise ValueError("q, k and v must be [tokens, heads, head_dim]")
    T = k.shape[0]
    if v.shape[0] != T or (q is not None and q.shape[0] != T):
        raise ValueError("q, k and v must hold the same number of tokens")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    kp, ks = _head_rows(k, "k", G, cfg)
    vp, vs = _head_rows(v, "v", G, cfg)
    qp, qs = _head_rows(q, "q", H, cfg) if q is not None else (None, 0)
    cache, B = _cache(cfg, k_pages, v_pages, page_table, kv_lens)
    st = _lib.tg_cache_append(
        qp, qs, kp, ks, vp, vs, _whole(q_offsets, "q_offsets", torch.int64, B + 1), T, cache, cfg.handle,
        _whole(q_out, "q_out", cfg.dtype, T * H * D) if q is not None else None,
        _whole(k_out, "k_out", cfg.dtype, T * G * D) if k_out is not None else None, _stream(stream))
    _check("tg_cache_append", st)


def tg_cache_read(offsets, kv_lens, page_table, k_pages, v_pages, cfg: AttnConfig, k=None, v=None, stream=None):
    """k and v [T, G, D] (or None), rows evenly spaced: the last offsets[b + 1] - offsets[b] tokens of every sequence b
    as the cache holds them; offsets int64 [B + 1]; the cache's tensors as tg_cache_append."""
    native = getattr(cfg, "_native", None)
    if native is not None:
        st = _binding.read(offsets, kv_lens, page_table, k_pages, v_pages, native, k, v,
                           None if stream is None else stream.cuda_stream)
        if st is not None:
            return _check("tg_cache_read", st)
    import torch
    G = cfg.num_kv_heads
    if k is None and v is None:
        raise ValueError("k or v is required")
    if any(t is not None and t.dim() != 3 for t in (k, v)):
        raise ValueError("k and v must be [tokens, heads, head_dim]")
    T = (v if k is None else k).shape[0]
    if v is not None and v.shape[0] != T:
        raise ValueError("k and v must hold the same number of tokens")
    kp, ks = _head_rows(k, "k", G, cfg) if k is not None else (None, 0)
    vp, vs = _head_rows(v, "v", G, cfg) if v is not None else (None, 0)
    cache, B = _cache(cfg, k_pages, v_pages, page_table, kv_lens)
    st = _lib.tg_cache_read(_whole(offsets, "offsets", torch.int64, B + 1), T, cache, cfg.handle, kp, ks, vp, vs, _stream(stream))
    _check("tg_cache_read", st)


def tg_attend_step(q, kv_lens, page_table, k_pages, v_pages, cfg: AttnConfig, out, out_lse=None, stream=None):
    """q and out [B, n, H, D]: the last n tokens of every sequence; out_lse f32 [B, n, H] or None; the cache's
    tensors as tg_cache_append."""
    native = getattr(cfg, "_native", None)
    if native is not None:
        st = _binding.step(q, kv_lens, page_table, k_pages, v_pages, native, out, out_lse,
                           None if stream is None else stream.cuda_stream)
        if st is not None:
            _check("tg_attend_step", st)
            return out
    import torch
    if q.dim() != 4:
        raise ValueError("q must be [batch, n, heads, head_dim]")
    B, n, H, D = q.shape
    cache, rows = _cache(cfg, k_pages, v_pages, page_table, kv_lens)
    if rows != B:
        raise ValueError("q holds %d sequences, page_table %d" % (B, rows))
    qp, qs = _head_rows(q, "q", cfg.num_heads, cfg)
    st = _lib.tg_attend_step(
        qp, qs, n, cache, cfg.handle, _whole(out, "out", cfg.dtype, B * n * H * D),
        _whole(out_lse, "out_lse", torch.float32, B * n * H) if out_lse is not None else None, _stream(stream))
    _check("tg_attend_step", st)
    return out


def tg_attend_shared(q, kv_lens, page_table, k_pages, v_pages, group_offsets, prefix_lens, cfg: AttnConfig, out, out_lse=None,
                     stream=None):
    """tg_attend_step for sequences that have a prefix in common: group_offsets int64 [groups + 1], group i is sequences
    group_offsets[i] .. group_offsets[i + 1] - 1; prefix_lens int32 [groups], the tokens that all of them begin with."""
    native = getattr(cfg, "_native", None)
    if native is not None:
        st = _binding.shared(q, kv_lens, page_table, k_pages, v_pages, group_offsets, prefix_lens, native, out, out_lse,
                             None if stream is None else stream.cuda_stream)
        if st is not None:
            _check("tg_attend_shared", st)
            return out
    import torch
    if q.dim() != 4:
        raise ValueError("q must be [batch, n, heads, head_dim]")
    B, n, H, D = q.shape
    if B * n > cfg.max_shared_tokens:
        raise ValueError("q holds %d tokens, the config's max_shared_tokens is %d" % (B * n, cfg.max_shared_tokens))
    cache, rows = _cache(cfg, k_pages, v_pages, page_table, kv_lens)
    if rows != B:
        raise ValueError("q holds %d sequences, page_table %d" % (B, rows))
    groups = prefix_lens.numel()
    qp, qs = _head_rows(q, "q", cfg.num_heads, cfg)
    st = _lib.tg_attend_shared(
        qp, qs, n, cache, _whole(group_offsets, "group_offsets", torch.int64, groups + 1),
        _whole(prefix_lens, "prefix_lens", torch.int32, groups), groups, cfg.handle, _whole(out, "out", cfg.dtype, B * n * H * D),
        _whole(out_lse, "out_lse", torch.float32, B * n * H) if out_lse is not None else None, _stream(stream))
    _check("tg_attend_shared", st)
    return out


def tg_attend_prompt(q, k, v, q_offsets, kv_offsets, cfg: AttnConfig, out, out_lse=None, causal=True, stream=None):
    """q and out [Tq, H, D], k and v [Tk, G, D]: sequences back to back, rows evenly spaced; q_offsets int64
    [B + 1]; kv_offsets int64 [B + 1] or None (as q_offsets); out_lse f32 [Tq, H] or None."""
    native = getattr(cfg, "_native", None)
    if native is not None:
        st = _binding.prompt(q, k, v, q_offsets, kv_offsets, native, out, out_lse, causal,
                             None if stream is None else stream.cuda_stream)
        if st is not None:
            _check("tg_attend_prompt", st)
            return out
    import torch
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, head_dim]")
    Tq, Tk, H, G = q.shape[0], k.shape[0], cfg.num_heads, cfg.num_kv_heads
    if v.shape[0] != Tk:
        raise ValueError("k and v must hold the same number of tokens")
    B = q_offsets.numel() - 1
    if B < 0:
        raise ValueError("q_offsets must hold batch + 1 values")
    qp, qs = _head_rows(q, "q", H, cfg)
    kp, ks = _head_rows(k, "k", G, cfg)
    vp, vs = _head_rows(v, "v", G, cfg)
    st = _lib.tg_attend_prompt(
        qp, qs, kp, ks, vp, vs, _whole(q_offsets, "q_offsets", torch.int64, B + 1),
        _whole(kv_offsets, "kv_offsets", torch.int64, B + 1) if kv_offsets is not None else None, B, Tq, Tk,
        1 if causal else 0, cfg.handle, _whole(out, "out", cfg.dtype, Tq * H * cfg.head_dim),
        _whole(out_lse, "out_lse", torch.float32, Tq * H) if out_lse is not None else None, _stream(stream))
    _check("tg_attend_prompt", st)
    return out


def tg_attn_status_word(cfg: AttnConfig) -> int:
    """The handle's sticky status bits (synchronous)."""
    f = c_uint32()
    _check("tg_attn_status_word", load_library().tg_attn_status_word(cfg.handle, ctypes.byref(f)))
    return int(f.value)


def tg_attn_clear_status(cfg: AttnConfig):
    _check("tg_attn_clear_status", load_library().tg_attn_clear_status(cfg.handle))
