"""Token generation with drafted windows, on a small random model of two layers: one KDA
layer (fp32 state pool) and one full-attention layer (e4m3 cache in pages).

A step takes each request's last token and its drafted ones through the model at
once, accepts a prefix of the drafts and draws the token after it:

  kda_decode            the window over a copy of the requests' states
  kda_cache_append      the window's K and V rows, quantised
  kda_paged_attention   the window over the cache
  kda_verify_draft      accepted drafts and the drawn token
  kda_decode            the accepted part once more, on the states themselves

The cache needs no second pass: rows of rejected drafts lie past the request's length
and the next window overwrites them.

    python examples/drafted_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import kda_decode_recurrence_gb300 as kda  # noqa: E402

DIM, VOCAB, DRAFTS = 256, 1000, 4
HEADS, K = 4, 128                 # KDA layer
QUERY, KEY, D, PAGE = 8, 2, 128, 16  # attention layer


class Model:
    def __init__(self, requests: int, pages_each: int, seed: int = 0, dev: str = "cuda"):
        g = torch.Generator(device=dev).manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, device=dev, generator=g) * shape[0] ** -0.5

        self.embed, self.head = weight(DIM, VOCAB).T.contiguous() * DIM ** 0.5, weight(DIM, VOCAB) * 2.5
        self.kda_in, self.kda_gate = weight(DIM, 3 * HEADS * K), weight(DIM, HEADS * K)
        self.kda_beta, self.kda_out = weight(DIM, HEADS), weight(HEADS * K, DIM) * 4
        self.attn_in, self.attn_out = weight(DIM, (QUERY + 2 * KEY) * D), weight(QUERY * D, DIM)
        self.a_log, self.dt_bias = torch.zeros(HEADS, device=dev), torch.zeros(HEADS, K, device=dev)
        # states: slots 0 .. requests - 1 are the requests', the next ones their copies
        self.pool = torch.zeros(2 * requests, HEADS, K, K, device=dev)
        self.slots = torch.arange(requests, dtype=torch.int32, device=dev)
        pages = requests * pages_each
        self.k_cache = torch.zeros(pages, KEY, PAGE, D, device=dev).to(torch.float8_e4m3fn)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.k_scale, self.v_scale = torch.ones(2, pages, KEY, PAGE, device=dev).unbind()
        self.table = torch.randperm(pages, device=dev, generator=g).to(torch.int32).view(requests, pages_each)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.generator, self.dev = g, dev

    def kda(self, x, cu, slots):
        """The KDA layer over packed tokens x; advances the slots' states."""
        T = x.shape[0]
        q, k, v = (x @ self.kda_in).to(torch.bfloat16).view(T, 3, HEADS, K).unbind(1)
        out = torch.empty(T, HEADS, K, device=self.dev)
        kda.kda_decode(out, q.contiguous(), k.contiguous(), v.contiguous(), (x @ self.kda_gate).view(T, HEADS, K),
                       (x @ self.kda_beta).contiguous(), self.a_log, self.dt_bias, cu, self.pool, slots,
                       gate_mode=kda.GATE_LOWER_BOUND, check_device=True)
        return x + out.view(T, -1) @ self.kda_out

    def attention(self, x, cu, lens, window):
        """The attention layer: the tokens' rows into the cache, then over it."""
        T = x.shape[0]
        qkv = (x @ self.attn_in).to(torch.bfloat16).view(T, QUERY + 2 * KEY, D)
        q, k, v = qkv.split([QUERY, KEY, KEY], dim=1)   # views: no copy is needed
        scales = dict(k_scale=self.k_scale, v_scale=self.v_scale)
        kda.kda_cache_append(self.k_cache, self.v_cache, k, v, cu, lens, self.table, **scales, check_device=True)
        out = torch.empty(T, QUERY, D, dtype=torch.bfloat16, device=self.dev)
        kda.kda_paged_attention(out, q, self.k_cache, self.v_cache, cu, lens, self.table, window, **scales,
                                check_device=True)
        return x + out.float().view(T, -1) @ self.attn_out

    def propose(self, last, n):
        """n drafted tokens per request and their probabilities: the model without its layers."""
        tokens, probs = [], []
        for _ in range(n):
            p = torch.softmax(self.embed[last.long()] @ self.head, -1)
            last = torch.multinomial(p, 1, generator=self.generator)[:, 0].to(torch.int32)
            tokens.append(last)
            probs.append(p)
        return torch.stack(tokens, 1), torch.stack(probs, 1)


def step(m: Model, last: torch.Tensor, n: int):
    """One step from each request's last token with n drafts.  Returns (tokens
    [B, n + 1], -1 past the drawn one; accepted [B]); states, cache and lengths advance."""
    B = last.shape[0]
    drafts, draft_probs = m.propose(last, n)
    window = torch.cat([last[:, None], drafts], 1)
    cu = torch.arange(B + 1, dtype=torch.int32, device=m.dev) * (n + 1)
    x = m.embed[window.flatten().long()]
    copies = m.slots + B
    m.pool[copies.long()] = m.pool[m.slots.long()]
    h = m.kda(x, cu, copies)
    lens = m.lens + n + 1
    h = m.attention(h, cu, lens, n + 1)
    probs = torch.softmax(h @ m.head, -1)
    tokens = torch.empty(B * (n + 1), dtype=torch.int32, device=m.dev)
    accepted = torch.empty(B, dtype=torch.int32, device=m.dev)
    uniform = torch.rand(B * (n + 1), device=m.dev, generator=m.generator)
    kda.kda_verify_draft(tokens, accepted, probs, draft_probs.reshape(B * n, -1), drafts.flatten().contiguous(),
                         uniform[:B * n], uniform[B * n:], torch.arange(B + 1, dtype=torch.int32, device=m.dev) * n,
                         check_device=True)
    # the states advance by the last token and the accepted drafts only
    kept = accepted + 1
    rows = (torch.arange(n + 1, device=m.dev)[None] < kept[:, None]).flatten()
    cu_kept = torch.cat([kept.new_zeros(1), kept.cumsum(0, dtype=torch.int32)])
    m.kda(x[rows], cu_kept, m.slots)
    m.lens += kept
    return tokens.view(B, n + 1), accepted


def main():
    B, steps = 3, 6
    m = Model(B, pages_each=4)
    last = torch.tensor([1, 2, 3], dtype=torch.int32, device=m.dev)
    for i in range(steps):
        tokens, accepted = step(m, last, DRAFTS)
        last = tokens.gather(1, accepted[:, None].long())[:, 0].contiguous()
        print(f"step {i}: accepted {accepted.tolist()}, tokens {[[t for t in row if t >= 0] for row in tokens.tolist()]}")
    print(f"lengths {m.lens.tolist()}")


if __name__ == "__main__":
    main()
