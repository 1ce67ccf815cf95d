"""Inputs of the attention tests on the device, and their 64-bit results."""
import numpy as np

from oracle import attention_oracle as A


def torch_types():
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ids(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype)).cuda()


class Cache:
    """A paged cache whose unused places hold NaN (the largest code of an 8-bit
    cache), pages in random order, and the page table of `lens`."""

    def __init__(self, lens, heads, dim, kind, page, layout, seed, fill=True, spare=3, shared_pool=False):
        import torch
        rng = np.random.default_rng(seed)
        self.lens, self.kind, self.page, self.layout = np.asarray(lens), kind, page, layout
        need = -(-self.lens // page)
        total = int(need.sum()) + spare
        self.order = rng.permutation(total)
        most = max(1, int(need.max()) if len(need) else 1)
        self.table = np.full((len(self.lens), most), -1, np.int64)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = self.order[at:at + n]
            at += n
        shape = (page, heads, dim) if layout == "token" else (heads, page, dim)
        t = torch_types()[kind]
        if shared_pool:  # keys and values of a page next to each other
            pool = torch.full((total, 2) + shape, float("nan"), device="cuda").to(t)
            self.k, self.v = pool[:, 0], pool[:, 1]
        else:
            self.k = torch.full((total,) + shape, float("nan"), device="cuda").to(t)
            self.v = torch.full((total,) + shape, float("nan"), device="cuda").to(t)
        self.keys, self.values = [], []
        if fill:
            g = torch.Generator("cuda").manual_seed(seed)
            for b, n in enumerate(self.lens):
                pair = []
                for pages in (self.k, self.v):
                    x = torch.randn(int(n), heads, dim, generator=g, device="cuda")
                    x = (x * 20).to(t) if kind == "e4m3" else x.to(t)
                    pos = torch.arange(int(n), device="cuda")
                    pg = ids(self.table[b], np.int64)[pos // page] if n else pos
                    raw, y = (pages.view(torch.uint8), x.view(torch.uint8)) if kind == "e4m3" else (pages, x)
                    if layout == "token":
                        raw[pg, pos % page] = y
                    else:
                        raw[pg, :, pos % page] = y
                    pair.append(f64(x))
                self.keys.append(pair[0])
                self.values.append(pair[1])

    def device_table(self, extra=0):
        """int32 [B, max_pages], with a row stride that is not the row's length when extra > 0."""
        t = np.full((self.table.shape[0], self.table.shape[1] + extra), -1, np.int32)
        t[:, :self.table.shape[1]] = self.table
        return ids(t, np.int32)[:, :self.table.shape[1]] if extra else ids(t, np.int32)


def check_attention(got, want):
    """got: device tensors (out [R.., D], lse [R..]); want: rows of attend()."""
    out, lse = got
    o, tol, z, ztol = want
    g = f64(out).reshape(o.shape)
    bad = ~(np.abs(g - o) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(g - o) - tol)))
    if lse is not None:
        h = lse.double().cpu().numpy().reshape(z.shape)
        empty = np.isinf(z)
        assert np.array_equal(h[empty], z[empty])
        assert (np.abs(h[~empty] - z[~empty]) <= ztol[~empty]).all(), float(np.abs(h[~empty] - z[~empty]).max())


def step_reference(cache, q, n, rep, scale, kind, weights, k_scales=None, v_scales=None, lens=None):
    """Rows of [B, n, H] in order."""
    B, _, H, D = q.shape
    res = [np.zeros((B, n, H, D)), np.zeros((B, n, H, D)), np.zeros((B, n, H)), np.zeros((B, n, H))]
    lens = cache.lens if lens is None else lens
    for b in range(B):
        sees = lens[b] - n + 1 + np.arange(n)
        for h in range(H):
            g = h // rep
            k, v = cache.keys[b][:, g], cache.values[b][:, g]
            if k_scales is not None:
                k, v = k * np.float64(np.float32(k_scales[g])), v * np.float64(np.float32(v_scales[g]))
            r = A.attend(q[b, :, h], k, v, sees, scale, kind, weights)
            for dst, x in zip(res, r):
                dst[b, :, h] = x
    return res
