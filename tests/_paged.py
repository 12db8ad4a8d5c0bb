"""Plain 64-bit forms of the paged-cache, attention and draft-verification calls,
and builders of their inputs.  The forms follow include/kda.h position by position;
tolerances are derived from the roundings the calls are allowed:

  a value rounded to bf16 is off by at most U = 2^-8 of it, to fp32 by 2^-24
"""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn
U_BF16 = 2.0 ** -8
U_F32 = 2.0 ** -24


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 of fraction."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e.astype(float) - 7))
    v = np.where((e == 15) & (f == 7), np.nan, v)
    return np.where(c >> 7, -v, v)


E4M3_TABLE = e4m3_values()


def quantise(x: np.ndarray):
    """(codes, scales) of rows x [..., D] of fp32 values, by the formula of kda_cache_append."""
    x = x.astype(np.float32)
    most = np.abs(x).max(-1)
    fine = np.isfinite(x).all(-1)
    with np.errstate(all="ignore"):
        scale = np.where(most > 0, most / np.float32(448), np.float32(1)).astype(np.float32)
        y = (x / scale[..., None]).astype(np.float32).astype(np.float64)
    y = np.where(fine[..., None], y, 0.0)
    positive = E4M3_TABLE[:127]                    # 0 .. 448, ascending with the code
    a = np.minimum(np.abs(y), 448.0)
    lo = np.searchsorted(positive, a, side="right") - 1
    hi = np.minimum(lo + 1, 126)
    up = (a - positive[lo] > positive[hi] - a) | ((a - positive[lo] == positive[hi] - a) & (lo % 2 == 1))
    code = np.where(up, hi, lo).astype(np.uint8) | (np.signbit(y).astype(np.uint8) << 7)
    scale = np.where(fine, scale, np.float32(np.nan))
    return code, scale


def cumulative(n) -> list[int]:
    return [0] + list(np.cumsum(n).astype(int))


class Case:
    """New tokens and a paged cache on the device.  ``n`` new tokens, ``lens``
    positions in use per request; ``junk`` fills every row that no position in use
    owns (page tails, free pages, scales) with that value."""

    def __init__(self, n, lens, HKV, D, page, cache="bf16", seed=0, junk=float("nan"), spare=3,
                 extra_pages=1, dev="cuda", amplitude=1.0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.lens, self.HKV, self.D, self.page, self.cache = list(n), list(lens), HKV, D, page, cache
        self.B, self.T, self.dev = len(self.n), sum(self.n), dev
        need = [-(-max(x, 0) // page) for x in self.lens]
        self.max_pages = max(need + [1]) + extra_pages
        self.num_pages = sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        table = torch.full((self.B, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            at += k
        shape = (self.num_pages, HKV, page, D)
        used = torch.zeros(self.num_pages, page, dtype=torch.bool)
        for b, L in enumerate(self.lens):
            for i in range(need[b]):
                used[table[b, i], :min(page, max(L, 0) - i * page)] = True
        self.used = used[:, None, :].expand(self.num_pages, HKV, page)
        self.tensors = {}
        for name in ("k", "v"):
            x = torch.randn(shape, generator=g) * amplitude
            if cache == "bf16":
                x[~self.used] = junk
                self.tensors[name] = (x.to(torch.bfloat16).to(dev), None)
            else:
                code = (x * 100).clamp(-448, 448).to(E4M3)
                scale = torch.rand(shape[:3], generator=g) * 0.02 + 0.001
                code.view(torch.uint8)[~self.used] = 0x7F if junk != junk else 0x7E
                scale[~self.used] = junk
                self.tensors[name] = (code.to(dev), scale.to(dev))
        self.table = table.to(dev)
        self.cu = torch.tensor(cumulative(self.n), dtype=torch.int32, device=dev)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        self.gen = g

    def args(self):
        """k_cache, v_cache and the scales' keyword arguments."""
        return (self.tensors["k"][0], self.tensors["v"][0]), dict(k_scale=self.tensors["k"][1], v_scale=self.tensors["v"][1])

    def dense(self, name, b, table=None) -> torch.Tensor:
        """Request b's rows 0 .. lens[b] - 1 of K or V as [L, HKV, D] in 64 bits; a
        position without a page is a row of zeros."""
        x, scale = self.tensors[name]
        table = (self.table if table is None else table).cpu()
        rows = []
        for pos in range(max(self.lens[b], 0)):
            pg = int(table[b, pos // self.page])
            if not 0 <= pg < self.num_pages:
                rows.append(torch.zeros(self.HKV, self.D, dtype=torch.float64, device=x.device))
                continue
            r = x[pg, :, pos % self.page]
            r = r.double() if scale is None else r.float().double() * scale[pg, :, pos % self.page].double()[:, None]
            rows.append(r)
        return torch.stack(rows) if rows else torch.zeros(0, self.HKV, self.D, dtype=torch.float64, device=x.device)


def attention(case: Case, q: torch.Tensor, scale: float, causal=True, window=0, table=None):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits, [T, H, D] and [T, H].

    The tolerance counts, per row: the weights rounded to bf16 (U of sum P |v|), the
    output rounded to bf16 (U of it), the scores' fp32 sums ((D + 4) roundings of
    scale sum |q| |k| at most, which moves the weights by that relative amount, once
    in each numerator and once in the sum), the exponential's own error (2^-21) and
    the sum of the weights (one fp32 rounding per position at most)."""
    T, H, D = q.shape
    G = H // case.HKV
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    cu = cumulative(case.n)
    for b in range(case.B):
        L, n = case.lens[b], case.n[b]
        if L <= 0 or n == 0:
            continue
        k, v = case.dense("k", b, table), case.dense("v", b, table)
        j = torch.arange(L, device=q.device)
        for i in range(n):
            p = L - n + i
            if p < 0:
                continue
            see = torch.ones(L, dtype=torch.bool, device=q.device)
            if causal:
                see &= j <= p
            if window:
                see &= j > p - window
            if not bool(see.any()):
                continue
            t = cu[b] + i
            for h in range(H):
                kk, vv = k[see][:, h // G], v[see][:, h // G]
                qq = q[t, h].double()
                x = scale * (kk @ qq)
                top = x.max()
                w = torch.exp(x - top)
                P = w / w.sum()
                out[t, h] = P @ vv
                lse[t, h] = top + torch.log(w.sum())
                off = (D + 4) * U_F32 * abs(scale) * (kk.abs() @ qq.abs()).max() + x.abs().max() * 4 * U_F32 + 2.0 ** -21
                some = P @ vv.abs()
                tol[t, h] = (U_BF16 + 2 * off + len(x) * U_F32) * some + U_BF16 * out[t, h].abs()
                ltol[t, h] = off + len(x) * U_F32 + lse[t, h].abs() * 4 * U_F32
    return out, lse, tol, ltol


def verify(target, draft, draft_tokens, accept_u, sample_u, n):
    """(tokens, accepted) by the definition, with exact sums of integers: the
    probabilities are scaled by 2^60 (exact for fp32 values of at least 2^-36 or 0)."""
    V = target.shape[1]
    cu = cumulative(n)
    tokens, accepted = [], []
    for b, m in enumerate(n):
        j = 0
        while j < m:
            x = int(draft_tokens[cu[b] + j])
            if not 0 <= x < V:
                break
            p = float(target[cu[b] + b + j, x])
            q = 1.0 if draft is None else float(draft[cu[b] + j, x])
            if not float(accept_u[cu[b] + j]) * q < p:
                break
            j += 1
        w = target[cu[b] + b + j].astype(np.float64)
        if j < m:
            if draft is None:
                less = np.zeros(V)
                if 0 <= int(draft_tokens[cu[b] + j]) < V:
                    less[int(draft_tokens[cu[b] + j])] = 1.0
            else:
                less = draft[cu[b] + j].astype(np.float64)
            w = w - less
        w = np.where(w > 0, w, 0.0)
        weights = [int(y * 2.0 ** 60) for y in w]
        total = sum(weights)
        drawn = -1
        if total > 0:
            num, den = float(sample_u[b]).as_integer_ratio()
            run = 0
            for v, y in enumerate(weights):
                run += y
                if y:
                    drawn = v
                if run * den > num * total:
                    break
        accepted.append(j)
        tokens += [int(draft_tokens[cu[b] + i]) for i in range(j)] + [drawn] + [-1] * (m - j)
    return np.array(tokens, dtype=np.int32), np.array(accepted, dtype=np.int32)
