"""One attention layer and a vocabulary projection, decoded with the library:
prompts (whole or in chunks), single tokens, an assisted-generation step, and
a beam search whose beams share their prompt's pages.

    python examples/decode_step.py            # needs the GPU

Every position runs the same path as in a serving loop:

  prompts   tg_cache_append (rotate, write the cache) -> tg_attend_prompt -> logits -> tg_select
  a token   tg_cache_append -> tg_attend_step (n = 1) -> logits -> tg_select
  K guesses tg_cache_append -> tg_attend_step (n = K + 1) -> logits -> tg_verify
  a chunk   tg_cache_append -> tg_cache_read (all so far) -> tg_attend_prompt -> logits
  beams     tg_cache_append -> tg_attend_shared -> logits -> tg_beam_step

The cache is 16-bit, or i8 with scales that are computed as it is written.  The
weights are random; main() checks that verifying the tokens which single steps
produced accepts all of them.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import logits_processing_token_gb300 as tg  # noqa: E402

HEADS, KV_HEADS, DIM, HIDDEN, VOCAB, PAGE = 8, 2, 64, 256, 1000, 16


class Layer:
    """Embedding, one attention layer, vocabulary projection; its paged cache (cache_dtype None: 16-bit, or "i8")."""

    def __init__(self, batch, max_len, seed=0, cache_dtype=None, shared_tokens=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[0] ** -0.5).bfloat16()

        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda").bfloat16()
        self.w_qkv = weight(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM)
        self.w_out, self.w_vocab = weight(HEADS * DIM, HIDDEN), weight(HIDDEN, VOCAB)
        inv_freq = 10000.0 ** (-torch.arange(0, DIM, 2) / DIM)
        self.attn = tg.AttnConfig(num_heads=HEADS, num_kv_heads=KV_HEADS, head_dim=DIM, page_size=PAGE, rotary_dim=DIM,
                                  inv_freq=inv_freq.tolist(), cache_dtype=cache_dtype, max_shared_tokens=shared_tokens)
        pages = -(-max_len // PAGE)
        page = (self.attn.page_bytes,) if cache_dtype == "i8" else self.attn.page_shape
        self.k_pages = torch.zeros(batch * pages, *page, dtype=self.attn.cache_dtype, device="cuda")
        self.v_pages = torch.zeros_like(self.k_pages)
        order = torch.randperm(batch * pages, generator=g, device="cuda")
        self.table = order.view(batch, pages).to(torch.int32)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.batch = batch

    def _append(self, ids, counts):
        """Project the new tokens, rotate them and write them into the cache."""
        x = self.embed[ids.long()]
        q, k, v = (t.unflatten(1, (-1, DIM)) for t in
                   (x @ self.w_qkv).split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], dim=1))
        offsets = torch.zeros(self.batch + 1, dtype=torch.int64, device="cuda")
        offsets[1:] = counts.cumsum(0)
        self.lens += counts.to(torch.int32)
        q_out, k_out = (torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k))
        tg.tg_cache_append(q, k, v, offsets, self.lens, self.table, self.k_pages, self.v_pages, self.attn, q_out, k_out)
        return x, q_out, k_out, v, offsets

    def _logits(self, x, attended):
        return ((x + attended.flatten(1) @ self.w_out) @ self.w_vocab).float()

    def prompts(self, ids, counts):
        """Logits after each prompt (packed ids, counts per prompt)."""
        x, q, k, v, offsets = self._append(ids, counts)
        out = torch.empty_like(q)
        tg.tg_attend_prompt(q, k, v, offsets, None, self.attn, out)
        last = offsets[1:] - 1
        return self._logits(x[last], out[last])

    def chunk(self, ids, counts):
        """prompts() for the next counts tokens of every prompt, after what the cache holds of it."""
        x, q, _, _, offsets = self._append(ids, counts)
        held = torch.zeros(self.batch + 1, dtype=torch.int64, device="cuda")
        held[1:] = self.lens.cumsum(0)
        k, v = (torch.empty(int(held[-1]), KV_HEADS, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        tg.tg_cache_read(held, self.lens, self.table, self.k_pages, self.v_pages, self.attn, k, v)
        out = torch.empty_like(q)
        tg.tg_attend_prompt(q, k, v, offsets, held, self.attn, out)
        last = offsets[1:] - 1
        return self._logits(x[last], out[last])

    def fork(self, prompt_len):
        """Every sequence begins with sequence 0's first prompt_len tokens: on the same pages as far as those are
        whole, and a copy of the page in which they end."""
        whole = prompt_len // PAGE
        self.table[1:, :whole] = self.table[0, :whole]
        if prompt_len % PAGE:
            for pages in (self.k_pages, self.v_pages):
                pages[self.table[1:, whole].long()] = pages[int(self.table[0, whole])].clone()
        self.lens.fill_(prompt_len)
        self.groups = torch.tensor([0, self.batch], device="cuda")
        self.prefix = torch.tensor([prompt_len], dtype=torch.int32, device="cuda")

    def reorder(self, prompt_len, parents):
        """Sequence b continues what sequence parents[b] holds: its pages behind the prompt's whole ones are copied."""
        own = slice(prompt_len // PAGE, None)
        for pages in (self.k_pages, self.v_pages):
            pages[self.table[:, own].long()] = pages[self.table[parents, own].long()].clone()

    def beam_step(self, ids):
        """ids [batch]: logits [batch, VOCAB] after one new token of every beam of one prompt (after fork())."""
        counts = torch.ones(self.batch, dtype=torch.int64, device="cuda")
        x, q, _, _, _ = self._append(ids, counts)
        q = q.view(self.batch, 1, HEADS, DIM)
        out = torch.empty_like(q)
        tg.tg_attend_shared(q, self.lens, self.table, self.k_pages, self.v_pages, self.groups, self.prefix, self.attn, out)
        return self._logits(x, out.flatten(0, 1).flatten(1).view(self.batch, HEADS, DIM))

    def step(self, ids):
        """ids [batch, n]: logits [batch, n, VOCAB] after each of the n new tokens."""
        n = ids.shape[1]
        counts = torch.full((self.batch,), n, dtype=torch.int64, device="cuda")
        x, q, _, _, _ = self._append(ids.reshape(-1), counts)
        q = q.view(self.batch, n, HEADS, DIM)
        out = torch.empty_like(q)
        tg.tg_attend_step(q, self.lens, self.table, self.k_pages, self.v_pages, self.attn, out)
        return self._logits(x, out.flatten(0, 1)).view(self.batch, n, VOCAB)


def pick(cfg, logits, tokens, lens, prompt_lens):
    """tg_select over rows whose histories are tokens[b, :lens[b]]."""
    B = logits.shape[0]
    offsets = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = lens.cumsum(0)
    history = tokens[torch.arange(tokens.shape[1], device="cuda") < lens[:, None]]
    out = torch.empty(B, dtype=torch.int32, device="cuda")
    tg.tg_select(logits, history, offsets, prompt_lens, cfg, None, out)
    return out


def run(batch=3, new_tokens=6, seed=0):
    """Decode new_tokens greedily, then check them with one verify step.
    Returns (tokens [batch, new_tokens], matches [batch])."""
    g = torch.Generator("cuda").manual_seed(seed + 1)
    counts = torch.tensor([5 + 20 * b for b in range(batch)], device="cuda")
    ids = torch.randint(0, VOCAB, (int(counts.sum()),), generator=g, device="cuda", dtype=torch.int32)
    cfg = tg.Config(vocab=VOCAB, mode="greedy", max_batch=batch)
    longest = int(counts.max()) + new_tokens + 1
    layer = Layer(batch, longest, seed)
    tokens = torch.zeros(batch, longest, dtype=torch.int32, device="cuda")
    tokens[torch.arange(longest, device="cuda") < counts[:, None]] = ids
    lens, plens = counts.clone(), counts.to(torch.int32)

    token = pick(cfg, layer.prompts(ids, counts), tokens, lens, plens)
    decoded = [token]
    for _ in range(new_tokens - 1):
        tokens[torch.arange(batch, device="cuda"), lens] = token
        lens += 1
        token = pick(cfg, layer.step(token[:, None])[:, 0].contiguous(), tokens, lens, plens)
        decoded.append(token)
    decoded = torch.stack(decoded, 1)

    # the same tokens as an assistant's guesses: the first is known, the rest are checked at once
    layer.lens.copy_(plens)
    K = new_tokens - 1
    logits = layer.step(decoded)
    matches = torch.empty(batch, dtype=torch.int32, device="cuda")
    chosen = torch.empty(batch, K + 1, dtype=torch.int32, device="cuda")
    tg.tg_verify(logits, decoded[:, 1:].contiguous(), K, cfg, None, matches, chosen)
    return decoded, matches


def beam_search(prompt, beams=4, new_tokens=6, seed=0, cache_dtype=None):
    """Beam search over one prompt (ids int32 [n], longer than 8 tokens), written in two chunks.
    Returns (tokens [beams, new_tokens], scores [beams]), best first."""
    n = prompt.numel()
    layer = Layer(beams, n + new_tokens, seed, cache_dtype, shared_tokens=beams)
    cfg = tg.Config(vocab=VOCAB, mode="greedy", max_batch=beams)
    keep = tg.tg_beam_keep(cfg, beams)
    counts = torch.zeros(beams, dtype=torch.int64, device="cuda")
    for part in (prompt[:8], prompt[8:]):  # (the other sequences have no tokens yet)
        counts[0] = part.numel()
        logits = layer.chunk(part, counts)[:1].expand(beams, VOCAB).contiguous()
    layer.fork(n)
    scores = torch.full((beams,), -1e9, device="cuda")
    scores[0] = 0.0  # at the first step all beams are the same: one of them counts
    tokens = torch.zeros(beams, 0, dtype=torch.int32, device="cuda")
    plens = torch.full((beams,), n, dtype=torch.int32, device="cuda")
    for i in range(new_tokens):
        history = torch.cat([prompt.expand(beams, n), tokens], 1)
        offsets = torch.arange(beams + 1, device="cuda") * history.shape[1]
        best = torch.empty(1, keep, device="cuda")
        ids, parents = (torch.empty(1, keep, dtype=torch.int32, device="cuda") for _ in range(2))
        tg.tg_beam_step(logits, scores, history.reshape(-1).contiguous(), offsets, plens, cfg, beams, best, ids, parents)
        chosen, parents, scores = ids[0, :beams].contiguous(), parents[0, :beams].long(), best[0, :beams].contiguous()
        tokens = torch.cat([tokens[parents], chosen[:, None]], 1)
        if i + 1 < new_tokens:
            layer.reorder(n, parents)
            logits = layer.beam_step(chosen)
    return tokens, scores


def main():
    prompt = torch.arange(40, dtype=torch.int32, device="cuda") * 7 % VOCAB
    for kind in (None, "i8"):
        print("beams", kind or "bf16", beam_search(prompt, cache_dtype=kind)[0][0].tolist())
    decoded, matches = run()
    print("decoded", decoded.tolist())
    print("guesses accepted", matches.tolist(), "of", decoded.shape[1] - 1)
    assert (matches == decoded.shape[1] - 1).all()


if __name__ == "__main__":
    main()
