"""Paged i8 caches of the tests: codes with a scale per token and key head, and what they stand for."""
import numpy as np

from tests.attention_util import Cache, f64, ids, step_reference

F32 = np.float32


def quantised(x):
    """(bytes, scales) of rows x [.., D] in f32, from the definition: every operation one f32 rounding."""
    x = np.asarray(x, F32)
    top = np.abs(x).max(-1)
    fine = np.isfinite(top)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        s = np.where(fine, top / F32(127), F32("nan")).astype(F32)
        q = np.where((s > 0)[..., None] & fine[..., None], x / s[..., None], F32(0))
    return (np.clip(np.rint(q), -127, 127) + 128).astype(np.uint8), s


def page_bytes(page, heads, dim, extra=0):
    return -(-page * heads * (dim + 4) // 16) * 16 + extra


def parts(pool, heads, dim, page, layout):
    """(codes in the layout, scales [pages, heads, page]) of a pool, as views."""
    n = page * heads
    codes = pool[:, :n * dim].unflatten(1, (page, heads, dim) if layout == "token" else (heads, page, dim))
    import torch
    return codes, pool[:, n * dim:n * (dim + 4)].view(torch.float32).unflatten(1, (heads, page))


class I8Cache(Cache):
    """Cache with i8 pages: unused places hold code 255 and a scale of NaN. extra: bytes behind each page."""

    def __init__(self, lens, heads, dim, page, layout, seed, fill=True, spare=3, extra=0, spread=1.0):
        import torch
        super().__init__(lens, heads, dim, "e4m3", page, layout, seed, fill=False, spare=spare)
        total = self.k.shape[0]
        self.kind, self.heads, self.dim = "i8", heads, dim
        pools = []
        for _ in range(2):
            p = torch.full((total, page_bytes(page, heads, dim, extra)), 255, dtype=torch.uint8, device="cuda")
            parts(p, heads, dim, page, layout)[1].fill_(float("nan"))
            pools.append(p)
        self.k, self.v = pools
        rng = np.random.default_rng(seed)
        if not fill:
            return
        for b, n in enumerate(self.lens):
            pos = np.arange(int(n))
            pg = self.table[b][pos // page]
            pair = []
            for pool in pools:
                x = rng.normal(0, 1, (int(n), heads, dim)).astype(F32) * np.exp(spread * rng.normal(0, 1, (int(n), heads, 1))).astype(F32)
                q, s = quantised(x)
                codes, scales = parts(pool, heads, dim, page, layout)
                pgd, sl = ids(pg, np.int64), ids(pos % page, np.int64)
                if layout == "token":
                    codes[pgd, sl] = torch.from_numpy(q).cuda()
                else:
                    codes[pgd, :, sl] = torch.from_numpy(q).cuda()
                scales[pgd, :, sl] = torch.from_numpy(s).cuda()
                pair.append((q.astype(np.float64) - 128) * s[..., None].astype(np.float64))
            self.keys.append(pair[0])
            self.values.append(pair[1])


def i8_reference(cache, q, n, rep, scale, kind, lens=None):
    """step_reference, for weights that are rounded to f16 relative to a scale of at most twice the largest of a value
    so far, the largest weight being at least 2^6 of such a unit (tensor memory kernel; 2^8 and the largest itself in the
    other): a weight below f16's normal numbers is off by half its smallest step, 2^-25, so by 2^-25 2^-6 times a value of
    at most twice the largest of the head, 2^-30 of that."""
    o, tol, z, ztol = step_reference(cache, q, n, rep, scale, kind, "f16", lens=lens)
    lens = cache.lens if lens is None else lens
    for b in range(q.shape[0]):
        for h in range(q.shape[2]):
            v = cache.values[b][:, h // rep]
            if v.size:
                tol[b, :, h] += min(int(lens[b]), len(v)) * 2.0 ** -30 * np.abs(v).max()
    return o, tol, z, ztol


def _tokens(cache, pool, b, pos, heads, dim):
    """Views of a pool and the indices of sequence b's tokens at pos: [(view, index), ..]."""
    page, slot = ids(cache.table[b][pos // cache.page], np.int64), ids(pos % cache.page, np.int64)
    import torch
    token = cache.layout == "token"
    if cache.kind == "i8":
        codes, scales = parts(pool, heads, dim, cache.page, cache.layout)
        return [(codes, (page, slot) if token else (page, slice(None), slot)), (scales, (page, slice(None), slot))]
    raw = pool.view(torch.uint8) if cache.kind == "e4m3" else pool
    return [(raw, (page, slot) if token else (page, slice(None), slot))]


def shared_cache(kind, members, prefix, lens, heads, dim, page, layout, seed, copies=False, **more):
    """A cache whose sequences begin, group by group, with the group's prefix: on the same pages as far as those are
    whole (copies: on pages of their own), behind that on their own. The first row of a group's table holds the whole
    prefix whatever its length."""
    lens = np.asarray(lens)
    first = np.repeat(np.concatenate([[0], np.cumsum(members)[:-1]]).astype(int), members)
    pre = np.repeat(np.asarray(prefix), members)
    alloc = np.where(first == np.arange(len(lens)), np.maximum(lens, pre), lens)
    alloc = np.where(np.repeat(members, members) == 1, lens, alloc)
    c = I8Cache(alloc, heads, dim, page, layout, seed, **more) if kind == "i8" else Cache(alloc, heads, dim, kind, page, layout, seed)
    for b in range(len(lens)):
        a, p = first[b], min(int(pre[b]), int(lens[b]))
        if a != b and p > 0:
            whole = 0 if copies else int(pre[b]) // page if lens[b] >= pre[b] // page * page else p // page
            pos = np.arange(whole * page, p)
            for pool in (c.k, c.v):
                for (view, src), (_, dst) in zip(_tokens(c, pool, a, pos, heads, dim), _tokens(c, pool, b, pos, heads, dim)):
                    if len(pos):
                        view[dst] = view[src]
            c.table[b, :whole] = c.table[a, :whole]
            for x in (c.keys, c.values):
                x[b][:p] = x[a][:p]
    c.lens = lens
    for x in (c.keys, c.values):
        for b, n in enumerate(lens):
            x[b] = x[b][:n]
    return c
