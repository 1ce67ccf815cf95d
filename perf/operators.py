"""The attention operators next to token selection, as cases that can be run and timed.

Three operators share one paged key-value cache:

- "append": rotate the new tokens' queries and keys by their positions and write the keys and
  values into the pages of the cache (tg_cache_append);
- "step": attention of the last n tokens of every sequence over the cache (tg_attend_step): n = 1 is a
  decode step, n = K + 1 the positions of an assisted-generation verify step;
- "prompt": causal attention over whole prompts, packed back to back (tg_attend_prompt).

`own` selects between the plain form (elementary torch operations in 32 bits, rounded once at the
end) and the calls of the library.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "e4m3": 1}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one sequence's new token: what a single interactive request pays per layer
        dict(name="append 1 token", op="append", heads=32, kv_heads=8, dim=128, type="bf16", cache="bf16", page=16,
             layout="token", rotary=128, pairs="halves", batch=1, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=1000, lens=1),
        # a decode step of a full batch into an 8-bit cache, contexts far out, odd rotation width
        dict(name="append 256 tokens e4m3", op="append", heads=32, kv_heads=8, dim=128, type="bf16", cache="e4m3", page=64,
             layout="head", rotary=64, pairs="neighbours", batch=256, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=131072, lens=2),
        # prompts of a prefill batch, some after a cached prefix
        dict(name="append prompts", op="append", heads=32, kv_heads=8, dim=128, type="bf16", cache="bf16", page=16,
             layout="token", rotary=128, pairs="halves", batch=12, new_lo=17, new_hi=2700, ctx_lo=0, ctx_hi=1500, lens=3),
        # one interactive request
        dict(name="step 1 x 4001", op="step", heads=32, kv_heads=8, dim=128, type="bf16", cache="bf16", page=16,
             layout="token", batch=1, new=1, len_lo=4001, len_hi=4001, lens=4),
        # a serving batch of mixed lengths, some slots of the batch empty
        dict(name="step 64 ragged", op="step", heads=32, kv_heads=8, dim=128, type="bf16", cache="bf16", page=16,
             layout="token", batch=64, new=1, len_lo=0, len_hi=4096, lens=5),
        # a full batch over an 8-bit cache
        dict(name="step 256 e4m3", op="step", heads=32, kv_heads=8, dim=128, type="bf16", cache="e4m3", page=64,
             layout="head", batch=256, new=1, len_lo=1, len_hi=2048, lens=6),
        # few long contexts, a key head for every query head
        dict(name="step 5 long f16", op="step", heads=16, kv_heads=16, dim=64, type="f16", cache="f16", page=32,
             layout="head", batch=5, new=1, len_lo=20000, len_hi=40000, lens=7),
        # assisted generation: 16 candidates and the token after them
        dict(name="step verify 32 x 17", op="step", heads=32, kv_heads=8, dim=128, type="bf16", cache="bf16", page=16,
             layout="token", batch=32, new=17, len_lo=256, len_hi=4096, lens=8),
        # one short prompt
        dict(name="prompt 61 f16", op="prompt", heads=12, kv_heads=12, dim=64, type="f16", batch=1, q_lo=61, q_hi=61,
             more_lo=0, more_hi=0, causal=True, lens=9),
        # a prefill batch of mixed lengths
        dict(name="prompt 64 ragged", op="prompt", heads=32, kv_heads=8, dim=128, type="bf16", batch=64, q_lo=1, q_hi=2048,
             more_lo=0, more_hi=0, causal=True, lens=10),
        # one long prompt
        dict(name="prompt 16384", op="prompt", heads=32, kv_heads=8, dim=128, type="bf16", batch=1, q_lo=16384, q_hi=16384,
             more_lo=0, more_hi=0, causal=True, lens=11),
        # chunks of prompts after what is already there; a head size that fills no tile, fewer keys than queries for some
        dict(name="prompt chunks f16 d80", op="prompt", heads=20, kv_heads=10, dim=80, type="f16", batch=9, q_lo=100, q_hi=1300,
             more_lo=-150, more_hi=2500, causal=True, lens=12),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    v = max(lo, min(hi, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    """One more case of the ranges above."""
    op = rng.choice(["append", "step", "step", "prompt", "prompt"])
    dim = rng.choice([64, 128, 128, 80, 96])
    kv = rng.choice([1, 2, 4, 8, 16])
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    while heads * dim > 5200 or heads * dim == 3072 or (heads + 2 * kv) * dim == 3072:
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 7])
    typ = rng.choice(["bf16", "bf16", "f16"])
    c = dict(op=op, heads=heads, kv_heads=kv, dim=dim, type=typ, lens=rng.randrange(1 << 30))
    if op != "prompt":
        c.update(cache=rng.choice([typ, typ, "e4m3"]), page=rng.choice([8, 16, 32, 64, 128]),
                 layout=rng.choice(["token", "head"]))
    if op == "append":
        b = _log_int(rng, 1, 256)
        most = max(1, 16000 // b)
        hi = 1 if rng.random() < 0.5 else _log_int(rng, 1, most)
        ctx = _log_int(rng, 1, 100000)
        c.update(rotary=rng.choice([dim, dim // 2, 0]), pairs=rng.choice(["halves", "neighbours"]), batch=b,
                 new_lo=_log_int(rng, 1, hi), new_hi=hi, ctx_lo=rng.randrange(ctx), ctx_hi=ctx)
    elif op == "step":
        b = _log_int(rng, 1, 256)
        hi = _log_int(rng, 16, min(40000, max(16, 260000 // b)))
        c.update(batch=b, new=rng.choice([1, 1, 1, rng.randint(2, 17)]), len_lo=rng.randrange(hi), len_hi=hi)
    else:
        b = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(8000, int(16000 / math.sqrt(b))))
        more = rng.choice([0, 0, _log_int(rng, 1, min(4000, int(8000 / math.sqrt(b))))])
        c.update(batch=b, q_lo=rng.randint(1, hi), q_hi=hi, more_lo=-(more // 8), more_hi=more,
                 causal=rng.random() < 0.85)
    return c


def _between(case, lo, hi):
    """The case's lengths: ragged over [lo, hi], the longest of them present."""
    r = np.random.default_rng(case["lens"])
    n = r.integers(lo, hi + 1, case["batch"])
    n[int(r.integers(0, case["batch"]))] = hi
    return n.astype(np.int64)


def _append_lens(case):
    new = _between(case, case["new_lo"], case["new_hi"])
    ctx = _between(case, case["ctx_lo"], case["ctx_hi"])[::-1]
    return new, ctx + new


def _prompt_lens(case):
    q = _between(case, case["q_lo"], case["q_hi"])
    more = np.random.default_rng(case["lens"] + 1).integers(case["more_lo"], case["more_hi"] + 1, case["batch"])
    return q, np.maximum(q + more, 0)


def _pairs(q, k, causal):
    """Visible (query, key) pairs of a sequence of q queries, the last of k keys' positions."""
    if not causal:
        return int(q * k)
    first = k - q + 1  # keys that query 0 sees
    n = min(q, q + first - 1) if first < 1 else q
    return int(n * (max(first, 1) + k) // 2) if n > 0 and k > 0 else 0


def work(case):
    H, G, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        new, _ = _append_lens(case)
        t = int(new.sum())
        return {"bytes": 2 * t * D * (2 * H + 3 * G) + BYTES[case["cache"]] * t * D * 2 * G + 16 * case["batch"],
                "flops": 3 * t * (H + G) * case["rotary"]}
    if case["op"] == "step":
        n, lens = case["new"], _between(case, case["len_lo"], case["len_hi"])
        keys = int(lens.sum())
        seen = sum(_pairs(n, int(k), True) for k in lens)
        return {"bytes": 2 * keys * G * D * BYTES[case["cache"]] + 4 * case["batch"] * n * H * (D + 1), "flops": 4 * seen * H * D}
    q, k = _prompt_lens(case)
    seen = sum(_pairs(int(a), int(b), case["causal"]) for a, b in zip(q, k))
    return {"bytes": 2 * D * (2 * H * int(q.sum()) + 2 * G * int(k.sum())) + 4 * H * int(q.sum()), "flops": 4 * seen * H * D}


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _table(case, lens, gen, first=None):
    """Page numbers of every sequence, in an order that a pool in use has; pages before `first` (whose contents the
    call does not touch) are page 0, the unused end of a row is -1."""
    P, B = case["page"], case["batch"]
    have = -(-lens // P)
    skip = np.zeros(B, np.int64) if first is None else first // P
    count = int((have - skip).sum())
    order = torch.randperm(count + 1, generator=gen, device="cuda").cpu().numpy()
    table = np.full((B, max(1, int(have.max()))), -1, np.int32)
    col = np.arange(table.shape[1])[None]
    table[(col < skip[:, None])] = order[count]
    inside = (col >= skip[:, None]) & (col < have[:, None])
    table[inside] = order[:count]
    return torch.from_numpy(table).cuda(), count + 1


def _pool(case, pages, gen, fill):
    G, D, P = case["kv_heads"], case["dim"], case["page"]
    shape = (pages, P, G, D) if case["layout"] == "token" else (pages, G, P, D)
    return (_normal(gen, *shape) * fill).to(TYPES[case["cache"]])


def _scales(case, gen):
    """Per key head: what one unit of the 8-bit cache stands for."""
    if case["cache"] != "e4m3":
        return None, None
    s = 0.02 + 0.03 * torch.rand(2, case["kv_heads"], generator=gen, device="cuda")
    return s[0].contiguous(), s[1].contiguous()


def _frequencies(case):
    r = case["rotary"]
    return np.power(10000.0, -np.arange(0, r, 2, dtype=np.float64) / max(r, 1)).astype(np.float32)


def _handle(case, s):
    """What a program sets up once per model: head counts, types, rotation, scales."""
    import logits_processing_token_gb300 as tg
    host = lambda t: None if t is None else t.tolist()  # noqa: E731
    more = {}
    if case["op"] != "prompt":
        more = dict(cache_dtype=case["cache"], page_size=case["page"], page_layout=case["layout"],
                    k_scales=host(s["k_scale"]), v_scales=host(s["v_scale"]))
    if case["op"] == "append":
        more.update(rotary_dim=case["rotary"], rotary_interleaved=case["pairs"] == "neighbours",
                    inv_freq=_frequencies(case).tolist())
    return tg.AttnConfig(num_heads=case["heads"], num_kv_heads=case["kv_heads"], head_dim=case["dim"],
                         dtype=case["type"], **more)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    H, G, D, B, t = case["heads"], case["kv_heads"], case["dim"], case["batch"], TYPES[case["type"]]
    s = dict(case=case)
    offsets = lambda n: torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int64)).cuda()  # noqa: E731
    if case["op"] == "append":
        new, lens = _append_lens(case)
        T = int(new.sum())
        # the three parts of one projection's output, as a model hands them on
        qkv = _normal(gen, T, (H + 2 * G) * D).to(t)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, G * D, G * D], dim=1))
        s["table"], pages = _table(case, lens, gen, first=lens - new)
        s["k_scale"], s["v_scale"] = _scales(case, gen)
        s["k_pages"], s["v_pages"] = _pool(case, pages, gen, 1.0), _pool(case, pages, gen, 1.0)
        s["offsets"], s["lens"] = offsets(new), torch.from_numpy(lens.astype(np.int32)).cuda()
        s["q_out"], s["k_out"] = torch.empty(T, H, D, dtype=t, device="cuda"), torch.empty(T, G, D, dtype=t, device="cuda")
        s["inv_freq"] = torch.from_numpy(_frequencies(case)).cuda()
    elif case["op"] == "step":
        n, lens = case["new"], _between(case, case["len_lo"], case["len_hi"])
        s["q"] = (_normal(gen, B, n, H, D) * 2).to(t)
        s["table"], pages = _table(case, lens, gen)
        s["k_scale"], s["v_scale"] = _scales(case, gen)
        fill = 1.0 if case["cache"] != "e4m3" else 25.0
        s["k_pages"], s["v_pages"] = _pool(case, pages, gen, fill), _pool(case, pages, gen, fill)
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["out"] = torch.empty(B, n, H, D, dtype=t, device="cuda")
        s["lse"] = torch.empty(B, n, H, device="cuda")
    else:
        nq, nk = _prompt_lens(case)
        s["q"] = (_normal(gen, int(nq.sum()), H, D) * 2).to(t)
        kv = _normal(gen, max(1, int(nk.sum())), 2 * G * D).to(t)
        s["k"], s["v"] = (x.unflatten(1, (G, D)) for x in kv.split(G * D, dim=1))
        s["q_offsets"], s["k_offsets"] = offsets(nq), offsets(nk)
        s["longest"] = (int(nq.max()), int(nk.max()))
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
    s["handle"] = _handle(case, s) if own else None
    return s


# ---------------------------------------------------------------- the plain forms

def _place(offsets, total):
    """(sequence, place in it) of every packed token."""
    at = torch.arange(total, device=offsets.device)
    seq = torch.bucketize(at, offsets[1:], right=True)
    return seq, at - offsets[seq]


def _rotate(x, angle, rotary, pairs):
    """x [T, heads, D] in 32 bits; angle [T, rotary / 2] in 64."""
    if not rotary:
        return x
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r, rest = x[..., :rotary], x[..., rotary:]
    if pairs == "halves":
        a, b = r.chunk(2, dim=-1)
        r = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    return torch.cat([r, rest], dim=-1)


def _to_cache(x, scale, kind):
    if kind != "e4m3":
        return x.to(TYPES[kind])
    return (x / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _write(pages, page, slot, x, layout):
    raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
    if layout == "token":
        raw[page, slot] = x
    else:
        raw[page, :, slot] = x


def _plain_append(s):
    case = s["case"]
    T = s["q"].shape[0]
    seq, j = _place(s["offsets"], T)
    pos = s["lens"].long()[seq] - (s["offsets"][1:] - s["offsets"][:-1])[seq] + j
    angle = pos.double()[:, None] * s["inv_freq"].double()[None]
    q = _rotate(s["q"].float(), angle, case["rotary"], case["pairs"])
    k = _rotate(s["k"].float(), angle, case["rotary"], case["pairs"])
    page = s["table"][seq, pos // case["page"]].long()
    slot = pos % case["page"]
    _write(s["k_pages"], page, slot, _to_cache(k, s["k_scale"], case["cache"]), case["layout"])
    _write(s["v_pages"], page, slot, _to_cache(s["v"].float(), s["v_scale"], case["cache"]), case["layout"])
    return {"q": q.to(s["q"].dtype), "k": k.to(s["k"].dtype), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _softmax_product(scores, hidden, v):
    """(softmax(scores) v, log of the sum of exponentials) with the places in `hidden` left out."""
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    weight = scores.sub_(top).exp_()
    total = weight.sum(dim=-1, keepdim=True)
    out = torch.matmul(weight, v) / total.clamp(min=1e-30)
    return out, (top + total.log()).squeeze(-1)


def _gathered(pages, table, scale, case):
    G, D = case["kv_heads"], case["dim"]
    raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    x = raw[table.clamp(min=0).long()].view(pages.dtype).float()
    x = x.transpose(2, 3) if case["layout"] == "token" else x  # [B, pages, heads, slots, D]
    x = x.transpose(1, 2).reshape(table.shape[0], G, -1, D)
    return x if scale is None else x * scale[:, None, None]


def _plain_step(s):
    case = s["case"]
    B, n, H, D = s["q"].shape
    G = case["kv_heads"]
    k, v = _gathered(s["k_pages"], s["table"], s["k_scale"], case), _gathered(s["v_pages"], s["table"], s["v_scale"], case)
    q = s["q"].float().view(B, n, G, H // G, D).permute(0, 2, 3, 1, 4).reshape(B, G, -1, D)
    scores = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    sees = s["lens"].long()[:, None] - (n - 1) + torch.arange(n, device=q.device)  # [B, n] keys that a token sees
    hidden = torch.arange(k.shape[2], device=q.device) >= sees[..., None]
    out, lse = _softmax_product(scores.view(B, G, H // G, n, -1), hidden[:, None, None], v[:, :, None])
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B, n, H, D).to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(B, n, H)}


def _plain_prompt(s):
    case = s["case"]
    (T, H, D), G = s["q"].shape, case["kv_heads"]
    Lq, Lk = s["longest"]
    qo, ko = s["q_offsets"], s["k_offsets"]
    nq, nk = qo[1:] - qo[:-1], ko[1:] - ko[:-1]
    i, j = torch.arange(Lq, device=qo.device), torch.arange(Lk, device=qo.device)
    q = s["q"][(qo[:-1, None] + i).clamp(max=T - 1)].float()  # padded [B, Lq, H, D]
    q = q.unflatten(2, (G, H // G)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    at = (ko[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    k, v = s["k"][at].float().transpose(1, 2), s["v"][at].float().transpose(1, 2)
    scores = torch.matmul(q, k.transpose(-1, -2)).div_(math.sqrt(D)).unflatten(2, (H // G, Lq))
    hidden = (j >= nk[:, None])[:, None]
    if case["causal"]:
        hidden = hidden | (j > i[:, None] + (nk - nq)[:, None, None])
    out, lse = _softmax_product(scores, hidden[:, None, None], v[:, :, None])
    seq, place = _place(qo, T)
    return {"out": out.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, place].to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[seq, place]}


# ---------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _plain_append, "step": _plain_step, "prompt": _plain_prompt}[op](s)
    import logits_processing_token_gb300 as tg
    if op == "append":
        tg.tg_cache_append(s["q"], s["k"], s["v"], s["offsets"], s["lens"], s["table"], s["k_pages"], s["v_pages"],
                           s["handle"], s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "step":
        tg.tg_attend_step(s["q"], s["lens"], s["table"], s["k_pages"], s["v_pages"], s["handle"], s["out"], s["lse"])
    else:
        tg.tg_attend_prompt(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], s["handle"], s["out"], s["lse"],
                            causal=s["case"]["causal"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the definition in 64 bits

def _attend_one(q, k, v, limit):
    """q [R, D], k and v [L, D], limit [R]: query r sees keys 0 .. limit[r] - 1. In 64 bits."""
    out = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    for a in range(0, q.shape[0], 4096):
        lim = limit[a:a + 4096]
        most = int(lim.max())
        if most <= 0:
            continue
        x = q[a:a + 4096] @ k[:most].T / math.sqrt(q.shape[1])
        x[torch.arange(most, device=q.device)[None] >= lim[:, None]] = -math.inf
        z = torch.logsumexp(x, dim=1)
        seen = lim > 0
        w = torch.exp(x - torch.where(seen, z, torch.zeros_like(z))[:, None])
        out[a:a + 4096] = torch.where(seen[:, None], w @ v[:most], torch.zeros_like(out[a:a + 4096]))
        lse[a:a + 4096] = torch.where(seen, z, torch.full_like(z, -math.inf))
    return out, lse


def exact(case, seed):
    if work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    H, G, D, B = case["heads"], case["kv_heads"], case["dim"], case["batch"]
    if case["op"] == "append":
        new, lens = _append_lens(case)
        table = s["table"].cpu().numpy()
        pos = np.concatenate([np.arange(e - n, e) for n, e in zip(new, lens)])
        seq = np.repeat(np.arange(B), new)
        r = case["rotary"]
        a = torch.from_numpy(pos[:, None] * _frequencies(case).astype(np.float64)[None]).cuda()
        turn = torch.polar(torch.ones_like(a), a)[:, None]  # one unit complex number per token and pair

        def turned(x):
            x = x.double().clone()
            if r:
                if case["pairs"] == "halves":
                    z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
                    x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
                else:
                    x[..., :r] = torch.view_as_real(torch.view_as_complex(x[..., :r].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
            return x

        q, k, v = turned(s["q"]), turned(s["k"]), s["v"].double()
        page = torch.from_numpy(table[seq, pos // case["page"]].astype(np.int64)).cuda()
        slot = torch.from_numpy(pos % case["page"]).cuda()
        pools = []
        for pool, x, scale in ((s["k_pages"], k, s["k_scale"]), (s["v_pages"], v, s["v_scale"])):
            p = pool.double()
            p = p if case["layout"] == "token" else p.transpose(1, 2).contiguous()
            p[page, slot] = x if scale is None else (x / scale.double()[:, None]).clamp(-448, 448)
            pools.append(p if case["layout"] == "token" else p.transpose(1, 2))
        return {"q": q, "k": k, "k_pages": pools[0], "v_pages": pools[1]}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:-1], dtype=torch.float64, device="cuda")
    if case["op"] == "step":
        n, lens = case["new"], _between(case, case["len_lo"], case["len_hi"])
        for b in range(B):
            L = int(lens[b])
            t = s["table"][b, :-(-L // case["page"])].long()
            k, v = (p.view(torch.uint8)[t].view(p.dtype).double() if p.dtype == torch.float8_e4m3fn else p[t].double()
                    for p in (s["k_pages"], s["v_pages"]))
            if case["layout"] == "head":
                k, v = k.transpose(1, 2), v.transpose(1, 2)
            k, v = k.reshape(-1, G, D), v.reshape(-1, G, D)
            limit = (L - n + 1 + torch.arange(n, device="cuda")).repeat_interleave(H // G)
            for g in range(G):
                kk, vv = k[:, g], v[:, g]
                if s["k_scale"] is not None:
                    kk, vv = kk * s["k_scale"][g].double(), vv * s["v_scale"][g].double()
                heads = slice(g * (H // G), (g + 1) * (H // G))
                o, z = _attend_one(s["q"][b, :, heads].double().reshape(-1, D), kk, vv, limit)
                out[b, :, heads], lse[b, :, heads] = o.view(n, -1, D), z.view(n, -1)
        return {"out": out, "lse": lse}
    nq, nk = _prompt_lens(case)
    qo, ko = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    for b in range(B):
        i = torch.arange(int(nq[b]), device="cuda")
        limit = i + 1 + int(nk[b] - nq[b]) if case["causal"] else torch.full_like(i, int(nk[b]))
        for h in range(H):
            rows, keys = slice(int(qo[b]), int(qo[b + 1])), slice(int(ko[b]), int(ko[b + 1]))
            g = h // (H // G)
            out[rows, h], lse[rows, h] = _attend_one(s["q"][rows, h].double(), s["k"][keys, g].double(), s["v"][keys, g].double(), limit)
    return {"out": out, "lse": lse}
