"""Plain 64-bit forms of the latent-cache, latent-attention and tree-attention calls, and
builders of their inputs.  The forms follow include/kda.h; tolerances are derived from the
roundings the calls are allowed (see `softmax64`)."""
from __future__ import annotations

import math
import random

import torch

from _paged import U_BF16, U_F32, cumulative

LATENT, ROPE, ROW, HEAD = 512, 64, 576, 128
SCALE = (HEAD + ROPE) ** -0.5


class LatentCase:
    """New tokens and a paged latent cache on the device: ``n`` new tokens, ``lens`` positions in
    use per request; ``junk`` fills every row that no position in use owns."""

    def __init__(self, n, lens, page, seed=0, junk=float("nan"), spare=3, extra_pages=1, dev="cuda", amplitude=1.0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.lens, self.page = list(n), list(lens), page
        self.B, self.T = len(self.n), sum(self.n)
        need = [-(-max(x, 0) // page) for x in self.lens]
        self.max_pages, self.num_pages = max(need + [1]) + extra_pages, sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        table = torch.full((self.B, self.max_pages), -1, dtype=torch.int32)
        used = torch.zeros(self.num_pages, page, dtype=torch.bool)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            at += k
            for i in range(k):
                used[table[b, i], :min(page, self.lens[b] - i * page)] = True
        x = torch.randn(self.num_pages, page, ROW, generator=g) * amplitude
        x[~used] = junk
        self.used, self.cache = used, x.to(torch.bfloat16).to(dev)
        self.table = table.to(dev)
        self.cu = torch.tensor(cumulative(self.n), dtype=torch.int32, device=dev)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)

    def dense(self, b, table=None):
        """Request b's rows [L, 576] in 64 bits; a position without a page is a row of zeros."""
        t = (self.table if table is None else table)[b].cpu()
        L = max(self.lens[b], 0)
        rows = torch.zeros(L, ROW, dtype=torch.float64, device=self.cache.device)
        for i in range(-(-L // self.page)):
            lo, hi = i * self.page, min(L, (i + 1) * self.page)
            if 0 <= int(t[i]) < self.num_pages:
                rows[lo:hi] = self.cache[int(t[i]), :hi - lo].double()
        return rows


def trees(n, seed=0, reach=6):
    """Per request a list of the sets of nodes that each node sees: itself and its ancestors."""
    r = random.Random(seed)
    out = []
    for k in n:
        seen = []
        for i in range(k):
            parent = r.randint(max(-1, i - reach), i - 1)
            seen.append((seen[parent] if parent >= 0 else set()) | {i})
        out.append(seen)
    return out


def mask_of(tree, words, dev="cuda"):
    """The [T, words] int32 mask of `trees`' sets."""
    rows = [[sum(1 << (a - 32 * w) for a in seen if a // 32 == w) for w in range(words)]
            for nodes in tree for seen in nodes]
    return torch.tensor(rows, dtype=torch.int64).reshape(-1, words).to(torch.int32).to(dev)


def seen_by(n, L, causal=True, nodes=None, dev="cuda"):
    """[n, L]: the positions that the new tokens see (none for padding)."""
    j, p = torch.arange(L, device=dev), (L - n + torch.arange(n, device=dev))[:, None]
    if nodes is None:
        see = j[None] <= p if causal else torch.ones(n, L, dtype=torch.bool, device=dev)
    else:
        see = torch.zeros(n, L, dtype=torch.bool)
        see[:, :max(0, L - n)] = True
        for i, s in enumerate(nodes):
            for a in s:
                if a < n and L - n + a >= 0:
                    see[i, L - n + a] = True
        see = see.to(dev)
    return see & (p >= 0)


def softmax64(q, k, v, see, scale):
    """(out, lse, tolerances of both) of queries q [n, H, Dk] over keys k [L, H or 1, Dk] and values
    v [L, H or 1, Dv] where see [n, L], in 64 bits.

    The tolerance counts, per row: the weights rounded to bf16 (U of sum P |v|), the output rounded
    to bf16 (U of it), the scores' fp32 sums ((Dk + 4) roundings of scale sum |q| |k| at most, which
    moves the weights by that relative amount, once in each numerator and once in the sum), the
    scores' own roundings, the exponential's error (2^-21) and the sum of the weights (one fp32
    rounding per position at most)."""
    n, H, Dk = q.shape
    L, Dv = v.shape[0], v.shape[2]
    out = torch.zeros(n, H, Dv, dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    if L == 0 or n == 0:
        return out, lse, tol, ltol
    some_row = see.any(1)
    for h in range(H):
        # what a row does not see has no influence on it, whatever it holds
        kk, vv, qq = k[:, min(h, k.shape[1] - 1)], v[:, min(h, v.shape[1] - 1)], q[:, h].double()
        x = torch.where(see, scale * (qq @ kk.T), -math.inf)
        size = torch.where(see, abs(scale) * (qq.abs() @ kk.abs().T), 0.0).amax(1)
        top = x.amax(1)
        w = torch.exp(x - torch.where(some_row, top, 0.0)[:, None])
        total = w.sum(1)
        P = w / torch.where(some_row, total, 1.0)[:, None]
        safe = torch.where(see.any(0)[:, None], vv, 0.0)
        o, mass = P @ safe, P @ safe.abs()
        e = torch.where(some_row, top + torch.log(total), -math.inf)
        count = see.sum(1).double()
        off = (Dk + 4) * U_F32 * size + torch.where(see, x.abs(), 0.0).amax(1) * 4 * U_F32 + 2.0 ** -21
        out[:, h], lse[:, h] = o, e
        tol[:, h] = (U_BF16 + 2 * off + count * U_F32)[:, None] * mass + U_BF16 * o.abs()
        ltol[:, h] = torch.where(some_row, off + count * U_F32 + e.abs() * 4 * U_F32, 0.0)
    return out, lse, tol, ltol


def close(out, lse, want):
    """Both within their tolerances; rows that see nothing are zeros and -inf."""
    o, e, tol, ltol = want
    off = (out.double() - o).abs()
    assert bool((off <= tol).all()), f"off by {float((off / tol.clamp_min(1e-300)).max()):.3g} tolerances"
    empty = torch.isneginf(e)
    assert torch.equal(torch.isneginf(lse), empty) and bool((out[empty] == 0).all())
    off = (lse.double() - e)[~empty].abs()
    assert bool((off <= ltol[~empty]).all()), f"lse off by {float((off / ltol[~empty]).max()):.3g} tolerances"
