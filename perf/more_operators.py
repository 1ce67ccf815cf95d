"""A cache that is quantised as it is written, its reading back, and attention that shares a
long prefix, as cases that can be run and timed.

Four operators over one paged key-value cache:

- "write": rotate new tokens and write their keys and values into an 8-bit cache whose scales are
  computed as it is written, one per token and key head (tg_cache_append), and read them back as
  the cache holds them (tg_cache_read);
- "read": whole sequences of a cache as packed 16-bit keys and values (tg_cache_read), what a chunk
  of a prompt attends together with its own;
- "step": attention of the last n tokens of every sequence over the 8-bit cache (tg_attend_step);
- "shared": the same over groups of sequences that have a prefix in common, read once for all of a
  group (tg_attend_shared): the beams of a prompt, several draws from it, requests under one system prompt.

`own` selects between the plain form (elementary torch operations in 32 bits, rounded once at the
end) and the calls of the library.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "i8": torch.uint8}
BYTES = {"bf16": 2, "f16": 2, "e4m3": 1, "i8": 1}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one sequence's new token
        dict(name="write 1 token", op="write", heads=32, kv_heads=8, dim=128, type="bf16", cache="i8", page=16, layout="token",
             rotary=128, pairs="halves", batch=1, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=1000, lens=1),
        # a decode step of a full batch, contexts far out, a head size that fills no tile, half of it rotated
        dict(name="write 300 tokens f16", op="write", heads=20, kv_heads=5, dim=96, type="f16", cache="i8", page=64, layout="head",
             rotary=48, pairs="neighbours", batch=300, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=131072, lens=2),
        # prompts of a prefill batch, some after a cached prefix
        dict(name="write prompts", op="write", heads=32, kv_heads=8, dim=128, type="bf16", cache="i8", page=16, layout="token",
             rotary=128, pairs="halves", batch=9, new_lo=17, new_hi=1500, ctx_lo=0, ctx_hi=1500, lens=3),
        # one short sequence of a 16-bit cache, as many key heads as query heads
        dict(name="read 1 x 517 f16", op="read", heads=16, kv_heads=16, dim=64, type="f16", cache="f16", page=32, layout="head",
             batch=1, len_lo=517, len_hi=517, lens=4),
        # the sequences of a batch of chunks, out of the 8-bit cache
        dict(name="read 40 i8", op="read", heads=32, kv_heads=8, dim=128, type="bf16", cache="i8", page=16, layout="token",
             batch=40, len_lo=1, len_hi=6000, lens=5),
        # one interactive request
        dict(name="step 1 x 4001 i8", op="step", heads=32, kv_heads=8, dim=128, type="bf16", cache="i8", page=16, layout="token",
             batch=1, new=1, len_lo=4001, len_hi=4001, lens=6),
        # a full serving batch
        dict(name="step 256 i8", op="step", heads=32, kv_heads=8, dim=128, type="bf16", cache="i8", page=64, layout="head",
             batch=256, new=1, len_lo=0, len_hi=2048, lens=7),
        # assisted generation: 16 candidates and the token after them
        dict(name="step verify 32 x 17 i8", op="step", heads=32, kv_heads=8, dim=128, type="bf16", cache="i8", page=16, layout="token",
             batch=32, new=17, len_lo=256, len_hi=4096, lens=8),
        # the beams of one prompt
        dict(name="shared 4 beams", op="shared", heads=32, kv_heads=8, dim=128, type="bf16", cache="bf16", page=16, layout="token",
             groups=1, mem_lo=4, mem_hi=4, pre_lo=1021, pre_hi=1021, own_lo=1, own_hi=60, new=1, lens=9),
        # a beam search over a batch of prompts
        dict(name="shared 64 x 4 beams", op="shared", heads=32, kv_heads=8, dim=128, type="bf16", cache="bf16", page=16, layout="token",
             groups=64, mem_lo=4, mem_hi=4, pre_lo=100, pre_hi=4000, own_lo=1, own_hi=128, new=1, lens=10),
        # a serving batch under one system prompt, 8-bit cache
        dict(name="shared system prompt i8", op="shared", heads=32, kv_heads=8, dim=128, type="bf16", cache="i8", page=16, layout="token",
             groups=1, mem_lo=128, mem_hi=128, pre_lo=6000, pre_hi=6000, own_lo=1, own_hi=1000, new=1, lens=11),
        # draws from several prompts, verified five tokens at a time; some groups of one, some slots empty
        dict(name="shared verify 9 groups f16 d80", op="shared", heads=20, kv_heads=10, dim=80, type="f16", cache="f16", page=32,
             layout="head", groups=9, mem_lo=1, mem_hi=14, pre_lo=0, pre_hi=5000, own_lo=0, own_hi=700, new=5, lens=12),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    return max(lo, min(hi, v))


def draw(rng):
    """One more case of the ranges above."""
    op = rng.choice(["write", "read", "step", "step", "shared", "shared", "shared"])
    dim = rng.choice([64, 128, 128, 80, 96])
    kv = rng.choice([1, 2, 4, 8, 16])
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    while heads * dim > 5200:
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 7])
    typ = rng.choice(["bf16", "bf16", "f16"])
    cache = "i8" if op in ("write", "step") else rng.choice([typ, "i8", "e4m3"])
    c = dict(op=op, heads=heads, kv_heads=kv, dim=dim, type=typ, cache=cache, page=rng.choice([8, 16, 32, 64, 128]),
             layout=rng.choice(["token", "head"]), lens=rng.randrange(1 << 30))
    if op == "write":
        b = _log_int(rng, 1, 256)
        most = max(1, 8000 // b)
        hi = 1 if rng.random() < 0.5 else _log_int(rng, 1, most)
        ctx = _log_int(rng, 1, 100000)
        c.update(rotary=rng.choice([dim, dim // 2, 0]), pairs=rng.choice(["halves", "neighbours"]), batch=b,
                 new_lo=_log_int(rng, 1, hi), new_hi=hi, ctx_lo=rng.randrange(ctx), ctx_hi=ctx)
    elif op == "read":
        b = _log_int(rng, 1, 256)
        hi = _log_int(rng, 16, max(16, 120000 // b))
        c.update(batch=b, len_lo=rng.randrange(hi), len_hi=hi)
    elif op == "step":
        b = _log_int(rng, 1, 256)
        hi = _log_int(rng, 16, min(40000, max(16, 260000 // b)))
        c.update(batch=b, new=rng.choice([1, 1, 1, rng.randint(2, 17)]), len_lo=rng.randrange(hi), len_hi=hi)
    else:
        groups = _log_int(rng, 1, 64)
        members = _log_int(rng, 1, max(1, 128 // groups))
        room = 300000 // (groups * members)
        pre = _log_int(rng, 16, max(16, min(20000, room)))
        mine = _log_int(rng, 16, max(16, min(2000, room // 2)))
        c.update(groups=groups, mem_lo=rng.randint(1, members), mem_hi=members, pre_lo=rng.randrange(pre), pre_hi=pre,
                 own_lo=rng.choice([0, 1, mine // 2]), own_hi=mine, new=rng.choice([1, 1, 1, rng.randint(2, 9)]))
    return c


def _between(case, lo, hi, count, which=0):
    """Lengths, ragged over [lo, hi], the largest of them present."""
    r = np.random.default_rng(case["lens"] + which)
    n = r.integers(lo, hi + 1, count)
    n[int(r.integers(0, count))] = hi
    return n.astype(np.int64)


def _write_lens(case):
    new = _between(case, case["new_lo"], case["new_hi"], case["batch"])
    return new, _between(case, case["ctx_lo"], case["ctx_hi"], case["batch"], 1) + new


def _groups(case):
    """(members of every group, its prefix, every sequence's group, its length): a sequence without tokens of its
    own is an empty slot of the batch."""
    members = _between(case, case["mem_lo"], case["mem_hi"], case["groups"])
    prefix = _between(case, case["pre_lo"], case["pre_hi"], case["groups"], 1)
    group = np.repeat(np.arange(case["groups"]), members)
    mine = _between(case, case["own_lo"], case["own_hi"], len(group), 2)
    return members, prefix, group, np.where(mine > 0, prefix[group] + mine, 0)


def _lens(case):
    return _groups(case)[3] if case["op"] == "shared" else _between(case, case["len_lo"], case["len_hi"], case["batch"])


def _seen(n, lens):
    """Visible (query, key) pairs of the last n tokens of sequences of these lengths."""
    return int(sum(np.maximum(lens - n + 1 + j, 0).sum() for j in range(n)))


def work(case):
    H, G, D = case["heads"], case["kv_heads"], case["dim"]
    key = 2 * G * (D * BYTES[case["cache"]] + (4 if case["cache"] == "i8" else 0))  # bytes of a token in the cache
    if case["op"] == "write":
        new, _ = _write_lens(case)
        t = int(new.sum())
        # queries in and out, keys and values in and out, and into the cache
        return {"bytes": t * (4 * D * H + 8 * D * G + key) + 16 * case["batch"], "flops": 3 * t * (H + G) * case["rotary"]}
    if case["op"] == "read":
        t = int(_lens(case).sum())
        return {"bytes": t * (key + 4 * D * G), "flops": 2 * t * G * D if case["cache"] in ("i8", "e4m3") else 0}
    lens, n = _lens(case), case["new"]
    keys = int(lens.sum())
    if case["op"] == "shared":
        _, prefix, group, _ = _groups(case)
        used = np.minimum(prefix[group], lens)
        most = np.zeros(case["groups"], np.int64)
        np.maximum.at(most, group, used)
        keys += int(most.sum()) - int(used.sum())
    return {"bytes": keys * key + len(lens) * n * H * (4 * D + 4), "flops": 4 * _seen(n, lens) * H * D}


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _page_bytes(case):
    """An 8-bit page with its scales: the codes, then one f32 per key head and token."""
    codes = case["page"] * case["kv_heads"]
    return -(-(codes * case["dim"] + 4 * codes) // 16) * 16


def _pool(case, pages, gen):
    G, D, P = case["kv_heads"], case["dim"], case["page"]
    shape = (P, G, D) if case["layout"] == "token" else (G, P, D)
    if case["cache"] != "i8":
        return (_normal(gen, pages, *shape) * (25.0 if case["cache"] == "e4m3" else 1.0)).to(TYPES[case["cache"]])
    pool = torch.zeros(pages, _page_bytes(case), dtype=torch.uint8, device="cuda")
    x = _normal(gen, pages, *shape)
    s = x.abs().amax(dim=-1) / 127.0
    codes, scales = _parts(pool, case)
    codes.copy_((x / s[..., None]).round().clamp(-127, 127).add(128).to(torch.uint8))
    s = s * (0.5 + torch.rand(s.shape, generator=gen, device="cuda"))  # tokens of unlike size
    scales.copy_(s.transpose(1, 2) if case["layout"] == "token" else s)
    return pool


def _parts(pool, case):
    """(codes in the page's layout, scales [pages, heads, tokens]) of an 8-bit pool, as views."""
    G, D, P = case["kv_heads"], case["dim"], case["page"]
    n = P * G
    codes = pool[:, :n * D].unflatten(1, (P, G, D) if case["layout"] == "token" else (G, P, D))
    return codes, pool[:, n * D:n * (D + 4)].view(torch.float32).unflatten(1, (G, P))


def _scales(case, gen):
    """Per key head: what one unit of an e4m3 cache stands for."""
    if case["cache"] != "e4m3":
        return None, None
    s = 0.02 + 0.03 * torch.rand(2, case["kv_heads"], generator=gen, device="cuda")
    return s[0].contiguous(), s[1].contiguous()


def _table(case, lens, gen, first=None):
    """Page numbers of every sequence, in an order that a pool in use has; pages before `first` (whose contents the
    call does not touch) are page 0, the unused end of a row is -1."""
    P, B = case["page"], len(lens)
    have = -(-lens // P)
    skip = np.zeros(B, np.int64) if first is None else first // P
    count = int((have - skip).sum())
    order = torch.randperm(count + 1, generator=gen, device="cuda").cpu().numpy()
    table = np.full((B, max(1, int(have.max()))), -1, np.int32)
    col = np.arange(table.shape[1])[None]
    table[(col < skip[:, None])] = order[count]
    inside = (col >= skip[:, None]) & (col < have[:, None])
    table[inside] = order[:count]
    return table, count + 1


def _shared_table(case, gen):
    """The whole pages of a group's prefix are the same for all its sequences; the page in which it ends is each
    sequence's own copy. Returns the table, the number of pages, and (from, to) of the copies."""
    members, prefix, group, lens = _groups(case)
    P, B = case["page"], len(group)
    first = np.concatenate([[0], np.cumsum(members)[:-1]])[group]  # of every sequence's group
    whole = prefix[group] // P
    have = np.maximum(-(-lens // P), -(-prefix[group] // P))
    col = np.arange(max(1, int(have.max())))[None]
    mine = (col < have[:, None]) & ((col >= whole[:, None]) | (first == np.arange(B))[:, None])
    count = int(mine.sum())
    table = np.full(mine.shape, -1, np.int32)
    table[mine] = torch.randperm(count, generator=gen, device="cuda").cpu().numpy()
    table = np.where((col < whole[:, None]), table[first], table)
    part = np.nonzero((prefix[group] % P > 0) & (first != np.arange(B)))[0]
    return table.astype(np.int32), max(1, count), table[first[part], whole[part]], table[part, whole[part]]


def _frequencies(case):
    r = case["rotary"]
    return np.power(10000.0, -np.arange(0, r, 2, dtype=np.float64) / max(r, 1)).astype(np.float32)


def _handle(case, s):
    """What a program sets up once per model: head counts, types, rotation, scales."""
    import logits_processing_token_gb300 as tg
    host = lambda t: None if t is None else t.tolist()  # noqa: E731
    more = {}
    if case["op"] == "write":
        more.update(rotary_dim=case["rotary"], rotary_interleaved=case["pairs"] == "neighbours",
                    inv_freq=_frequencies(case).tolist())
    if case["op"] == "shared":
        more.update(max_shared_tokens=s["q"].shape[0] * s["q"].shape[1])
    return tg.AttnConfig(num_heads=case["heads"], num_kv_heads=case["kv_heads"], head_dim=case["dim"], dtype=case["type"],
                         cache_dtype=case["cache"], page_size=case["page"], page_layout=case["layout"],
                         k_scales=host(s["k_scale"]), v_scales=host(s["v_scale"]), **more)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    H, G, D, t = case["heads"], case["kv_heads"], case["dim"], TYPES[case["type"]]
    s = dict(case=case)
    offsets = lambda n: torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int64)).cuda()  # noqa: E731
    empty = lambda *shape, dtype=t: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    copies = None
    if case["op"] == "write":
        new, lens = _write_lens(case)
        T = int(new.sum())
        # the three parts of one projection's output, as a model hands them on; heads of unlike size, as keys have
        size = 0.2 + 2.0 * torch.rand(H + 2 * G, 1, generator=gen, device="cuda")
        qkv = (_normal(gen, T, H + 2 * G, D) * size).flatten(1).to(t)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, G * D, G * D], dim=1))
        table, pages = _table(case, lens, gen, first=lens - new)
        s["offsets"], s["q_out"] = offsets(new), empty(T, H, D)
        s["k_out"], s["v_out"] = empty(T, G, D), empty(T, G, D)
        s["inv_freq"] = torch.from_numpy(_frequencies(case)).cuda()
    elif case["op"] == "read":
        lens = _lens(case)
        table, pages = _table(case, lens, gen)
        s["offsets"] = offsets(lens)
        s["k_out"], s["v_out"] = empty(int(lens.sum()), G, D), empty(int(lens.sum()), G, D)
    else:
        n, lens = case["new"], _lens(case)
        if case["op"] == "shared":
            members, prefix, _, _ = _groups(case)
            s["groups"], s["prefix"] = offsets(members), torch.from_numpy(prefix.astype(np.int32)).cuda()
            table, pages, *copies = _shared_table(case, gen)
        else:
            table, pages = _table(case, lens, gen)
        s["q"] = (_normal(gen, len(lens), n, H, D) * 2).to(t)
        s["out"], s["lse"] = empty(len(lens), n, H, D), empty(len(lens), n, H, dtype=torch.float32)
    s["table"], s["lens"] = torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda()
    s["k_scale"], s["v_scale"] = _scales(case, gen)
    s["k_pages"], s["v_pages"] = _pool(case, pages, gen), _pool(case, pages, gen)
    if copies and len(copies[0]):
        src, dst = (torch.from_numpy(x.astype(np.int64)).cuda() for x in copies)
        for pool in (s["k_pages"], s["v_pages"]):
            raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
            raw[dst] = raw[src]
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


def _tokens(pool, page, slot, scale, case):
    """Single tokens out of a pool, in 32 bits: [T, heads, D]."""
    token = case["layout"] == "token"
    if case["cache"] == "i8":
        codes, scales = _parts(pool, case)
        x = codes[page, slot] if token else codes[page, :, slot]
        return (x.float() - 128.0) * scales[page, :, slot][..., None]
    raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
    x = (raw[page, slot] if token else raw[page, :, slot]).view(pool.dtype).float()
    return x if scale is None else x * scale[:, None]


def _keep(pool, page, slot, x, case):
    """x [T, heads, D] into an 8-bit pool, each head's scale its largest value over 127."""
    s = x.abs().amax(dim=-1) / 127.0
    q = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x)).round().clamp(-127, 127).add(128).to(torch.uint8)
    codes, scales = _parts(pool, case)
    if case["layout"] == "token":
        codes[page, slot] = q
    else:
        codes[page, :, slot] = q
    scales[page, :, slot] = s


def _plain_write(s):
    case = s["case"]
    t = s["q"].dtype
    seq, j = _place(s["offsets"], s["q"].shape[0])
    pos = s["lens"].long()[seq] - (s["offsets"][1:] - s["offsets"][:-1])[seq] + j
    angle = pos.double()[:, None] * s["inv_freq"].double()[None]
    q = _rotate(s["q"].float(), angle, case["rotary"], case["pairs"])
    k = _rotate(s["k"].float(), angle, case["rotary"], case["pairs"])
    page, slot = s["table"][seq, pos // case["page"]].long(), pos % case["page"]
    _keep(s["k_pages"], page, slot, k, case)
    _keep(s["v_pages"], page, slot, s["v"].float(), case)
    return {"q": q.to(t), "k": _tokens(s["k_pages"], page, slot, None, case).to(t),
            "v": _tokens(s["v_pages"], page, slot, None, case).to(t)}


def _plain_read(s):
    case, t = s["case"], s["k_out"].dtype
    seq, pos = _place(s["offsets"], s["k_out"].shape[0])
    page, slot = s["table"][seq, pos // case["page"]].long(), pos % case["page"]
    return {"k": _tokens(s["k_pages"], page, slot, s["k_scale"], case).to(t),
            "v": _tokens(s["v_pages"], page, slot, s["v_scale"], case).to(t)}


def _softmax_product(scores, hidden, v):
    """(softmax(scores) v, log of the sum of exponentials) with the places in `hidden` left out."""
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    weight = scores.sub_(top).exp_()
    total = weight.sum(dim=-1, keepdim=True)
    out = torch.matmul(weight, v) / total.clamp(min=1e-30)
    return out, (top + total.log()).squeeze(-1)


def _gathered(pool, table, scale, case):
    """Whole sequences out of a pool, in 32 bits: [B, heads, places, D]."""
    G, D = case["kv_heads"], case["dim"]
    at = table.clamp(min=0).long()
    if case["cache"] == "i8":
        codes, scales = _parts(pool, case)
        x = codes[at].float().sub_(128.0)
        s = scales[at]
        x = x.mul_((s.transpose(2, 3) if case["layout"] == "token" else s)[..., None])
    else:
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        x = raw[at].view(pool.dtype).float()
    x = x.transpose(2, 3) if case["layout"] == "token" else x  # [B, pages, heads, slots, D]
    x = x.transpose(1, 2).reshape(table.shape[0], G, -1, D)
    return x if scale is None else x * scale[:, None, None]


def _plain_attention(s):
    # A sequence's own row of the table names its whole prefix too: sharing changes what is read, not what comes out.
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


# ---------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "step": _plain_attention, "shared": _plain_attention}[op](s)
    import logits_processing_token_gb300 as tg
    cache = (s["lens"], s["table"], s["k_pages"], s["v_pages"])
    if op == "write":
        tg.tg_cache_append(s["q"], s["k"], s["v"], s["offsets"], *cache, s["handle"], s["q_out"])
        tg.tg_cache_read(s["offsets"], *cache, s["handle"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    if op == "read":
        tg.tg_cache_read(s["offsets"], *cache, s["handle"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "step":
        tg.tg_attend_step(s["q"], *cache, s["handle"], s["out"], s["lse"])
    else:
        tg.tg_attend_shared(s["q"], *cache, s["groups"], s["prefix"], s["handle"], s["out"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the definition in 64 bits

def _stored(pool, scale, case):
    """All that a pool stands for: [pages * tokens, heads, D] in 64 bits."""
    G, D, P = case["kv_heads"], case["dim"], case["page"]
    if case["cache"] == "i8":
        raw = pool.cpu().numpy()
        x = raw[:, :P * G * D].astype(np.float64) - 128.0
        x = x.reshape((-1, P, G, D) if case["layout"] == "token" else (-1, G, P, D))
        x = x if case["layout"] == "token" else x.swapaxes(1, 2)
        f = np.ascontiguousarray(raw[:, P * G * D:P * G * (D + 4)]).view(np.float32).reshape(-1, G, P).swapaxes(1, 2)
        return torch.from_numpy(np.ascontiguousarray(x * f[..., None].astype(np.float64)).reshape(-1, G, D)).cuda()
    x = pool.double()
    x = (x if case["layout"] == "token" else x.transpose(1, 2)).reshape(-1, G, D)
    return x if scale is None else x * scale.double()[:, None]


def _positions(table, lens, P):
    """Where the tokens of each sequence are in _stored."""
    return [(np.repeat(row[:-(-int(n) // P)].astype(np.int64), P) * P + np.tile(np.arange(P), -(-int(n) // P)))[:int(n)]
            for row, n in zip(table, lens)]


def exact(case, seed):
    s = prepare(case, seed)
    H, G, D = case["heads"], case["kv_heads"], case["dim"]
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    if case["op"] == "write":
        new, _ = _write_lens(case)
        pos = np.concatenate([np.arange(e - n, e) for n, e in zip(new, lens)])
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

        def kept(x):
            unit = x.abs().max(dim=-1, keepdim=True).values / 127
            return torch.round(x / unit.clamp(min=1e-300)) * unit

        return {"q": turned(s["q"]), "k": kept(turned(s["k"])), "v": kept(s["v"].double())}
    where = _positions(table, lens, case["page"])
    k, v = _stored(s["k_pages"], s["k_scale"], case), _stored(s["v_pages"], s["v_scale"], case)
    if case["op"] == "read":
        at = torch.from_numpy(np.concatenate(where)).cuda()
        return {"k": k[at], "v": v[at]}
    B, n = len(lens), case["new"]
    out = torch.zeros(B, n, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, n, H), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        at = torch.from_numpy(where[b]).cuda()
        kk, vv = k[at].transpose(0, 1), v[at].transpose(0, 1)  # [G, L, D]
        for j in range(n):
            sees = int(lens[b]) - n + 1 + j
            if sees <= 0:
                continue
            x = s["q"][b, j].double().view(G, H // G, D) @ kk[:, :sees].transpose(1, 2) / math.sqrt(D)
            z = torch.logsumexp(x, dim=-1)
            lse[b, j] = z.reshape(H)
            out[b, j] = (torch.exp(x - z[..., None]) @ vv[:, :sees]).reshape(H, D)
    return {"out": out, "lse": lse}
