"""One attention layer and a vocabulary projection, decoded with the library:
prompts, single tokens, and an assisted-generation step.

    python examples/decode_step.py            # needs the GPU

Every position runs the same path as in a serving loop:

  prompts   tg_cache_append (rotate, write the cache) -> tg_attend_prompt -> logits -> tg_select
  a token   tg_cache_append -> tg_attend_step (n = 1) -> logits -> tg_select
  K guesses tg_cache_append -> tg_attend_step (n = K + 1) -> logits -> tg_verify

The weights are random; main() checks that verifying the tokens which single
steps produced accepts all of them.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import logits_processing_token_gb300 as tg  # noqa: E402

HEADS, KV_HEADS, DIM, HIDDEN, VOCAB, PAGE = 8, 2, 64, 256, 1000, 16


class Layer:
    """Embedding, one attention layer, vocabulary projection; its paged cache."""

    def __init__(self, batch, max_len, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[0] ** -0.5).bfloat16()

        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda").bfloat16()
        self.w_qkv = weight(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM)
        self.w_out, self.w_vocab = weight(HEADS * DIM, HIDDEN), weight(HIDDEN, VOCAB)
        inv_freq = 10000.0 ** (-torch.arange(0, DIM, 2) / DIM)
        self.attn = tg.AttnConfig(num_heads=HEADS, num_kv_heads=KV_HEADS, head_dim=DIM, page_size=PAGE, rotary_dim=DIM,
                                  inv_freq=inv_freq.tolist())
        pages = -(-max_len // PAGE)
        self.k_pages = torch.zeros(batch * pages, PAGE, KV_HEADS, DIM, dtype=torch.bfloat16, device="cuda")
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


def main():
    decoded, matches = run()
    print("decoded", decoded.tolist())
    print("guesses accepted", matches.tolist(), "of", decoded.shape[1] - 1)
    assert (matches == decoded.shape[1] - 1).all()


if __name__ == "__main__":
    main()
