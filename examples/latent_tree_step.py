"""A layer of latent attention through a prompt and through steps with drafted trees, on random
weights.

  kda_latent_append     every token's latent row (normed) into a paged cache
  kda_latent_expanded   the prompts' tokens, over keys and values expanded from their rows
  kda_latent_attention  a tree of drafted tokens over the cache, heads absorbed into the latents
  (a path of the tree is accepted; its rows are appended once more, one behind the other)

A node of the tree sees the cached text and its ancestors.  Its position is not its row's in the
cache but its depth in the tree, which the position part of rows and queries says (here: a
rotation by the depth).

    python examples/latent_tree_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import kda_decode_recurrence_gb300 as kda  # noqa: E402

DIM, HEADS, PAGE = 256, 16, 16
NOPE, ROPE, LATENT = kda.EXPANDED, kda.LATENT_ROPE, kda.LATENT


def rotate(x, pos):
    """The position part x [T, .., ROPE] rotated by each token's position."""
    half = ROPE // 2
    angle = pos.double()[:, None] * 100.0 ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    angle = angle.view(len(pos), *[1] * (x.dim() - 2), half)
    a, b = x.double().split(half, -1)
    return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)


class Layer:
    def __init__(self, requests: int, pages_each: int, seed: int = 0, dev: str = "cuda"):
        g = torch.Generator(device=dev).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, device=dev, generator=g) * shape[-2] ** -0.5).to(torch.bfloat16)

        self.w_q, self.w_latent = weight(DIM, HEADS * (NOPE + ROPE)), weight(DIM, LATENT + ROPE)
        self.gamma = 1 + 0.1 * torch.randn(LATENT, device=dev, generator=g)
        self.w_k, self.w_v = weight(HEADS, LATENT, NOPE), weight(HEADS, LATENT, NOPE)  # latents to keys, values
        pages = requests * pages_each
        self.cache = torch.zeros(pages, PAGE, LATENT + ROPE, dtype=torch.bfloat16, device=dev)
        self.table = torch.randperm(pages, device=dev, generator=g).to(torch.int32).view(requests, pages_each)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.dev = dev

    def project(self, x, pos):
        """Queries [T, HEADS, 128 + 64] and latent rows [T, 576] (not normed) of hidden rows x."""
        T = x.shape[0]
        q = (x @ self.w_q).view(T, HEADS, NOPE + ROPE)
        q = torch.cat([q[..., :NOPE], rotate(q[..., NOPE:], pos).to(q.dtype)], -1)
        rows = x @ self.w_latent
        return q, torch.cat([rows[:, :LATENT], rotate(rows[:, LATENT:], pos).to(rows.dtype)], -1)

    def append(self, rows, cu, lens):
        kda.kda_latent_append(self.cache, rows, cu, lens, self.table, gamma=self.gamma, check_device=True)

    def rows_of(self, b, n):
        """The cached rows of request b's first n positions."""
        pos = torch.arange(n, device=self.dev)
        return self.cache[self.table[b].long()[pos // PAGE], pos % PAGE]

    def prompt(self, x, n):
        """Prompts of n[b] tokens each; returns their heads' outputs [T, HEADS, 128]."""
        pos = torch.cat([torch.arange(k, device=self.dev) for k in n])
        cu = torch.tensor([0, *torch.tensor(n).cumsum(0).tolist()], dtype=torch.int32, device=self.dev)
        q, rows = self.project(x, pos)
        self.lens = torch.tensor(n, dtype=torch.int32, device=self.dev)
        self.append(rows, cu, self.lens)
        rows = torch.cat([self.rows_of(b, k) for b, k in enumerate(n)])         # normed, as every later step sees them
        kv = torch.einsum("tc,hcd->thd", rows[:, :LATENT], torch.cat([self.w_k, self.w_v], -1))
        out = torch.empty(len(pos), HEADS, NOPE, dtype=torch.bfloat16, device=self.dev)
        kda.kda_latent_expanded(out, q, kv.contiguous(), rows[:, LATENT:], cu, cu, check_device=True)
        return out

    def tree(self, x, parents):
        """Trees of drafted tokens, parents[b][i] the parent of node i (-1: the cached text).  Returns the heads'
        outputs [T, HEADS, 128]; the nodes' rows lie behind the text, whose lengths stay as they are."""
        most = max(len(p) for p in parents)
        mask, depth = [], []
        for p in parents:
            seen, level = [], []
            for i, parent in enumerate(p):
                seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
                level.append(level[parent] + 1 if parent >= 0 else 0)
            mask += [[s >> 32 * w & 0xFFFFFFFF for w in range(-(-most // 32))] for s in seen]
            depth += level
        n = torch.tensor([len(p) for p in parents], dtype=torch.int32, device=self.dev)
        cu = torch.cat([n.new_zeros(1), n.cumsum(0, dtype=torch.int32)])
        pos = torch.tensor(depth, device=self.dev) + self.lens.repeat_interleave(n)
        q, rows = self.project(x, pos)
        self.append(rows, cu, self.lens + n)
        absorbed = torch.cat([torch.einsum("thd,hcd->thc", q[..., :NOPE], self.w_k), q[..., NOPE:]], -1).contiguous()
        sums = torch.empty(len(pos), HEADS, LATENT, dtype=torch.bfloat16, device=self.dev)
        bits = torch.tensor(mask, dtype=torch.int64, device=self.dev).to(torch.int32)
        kda.kda_latent_attention(sums, absorbed, self.cache, cu, self.lens + n, self.table, tree_mask=bits,
                                 check_device=True)
        return torch.einsum("thc,hcd->thd", sums, self.w_v)

    def accept(self, x, paths):
        """The hidden rows x of each request's accepted path (paths[b] of them), one behind the other."""
        n = torch.tensor(paths, dtype=torch.int32, device=self.dev)
        cu = torch.cat([n.new_zeros(1), n.cumsum(0, dtype=torch.int32)])
        pos = torch.cat([torch.arange(int(L), int(L) + k, device=self.dev) for L, k in zip(self.lens, paths)])
        self.lens = self.lens + n
        self.append(self.project(x, pos)[1], cu, self.lens)


def main():
    g = torch.Generator(device="cuda").manual_seed(1)
    layer, n = Layer(2, pages_each=8), [40, 23]
    out = layer.prompt(torch.randn(sum(n), DIM, device="cuda", generator=g).to(torch.bfloat16), n)
    print(f"prompts of {n} tokens: outputs {tuple(out.shape)}, norm {float(out.float().norm()):.2f}")
    parents = [[-1, 0, 0, 1, 1, 2], [-1, -1, 0, 2]]
    paths = [[0, 1, 4], [0, 2, 3]]
    for i in range(3):
        x = torch.randn(10, DIM, device="cuda", generator=g).to(torch.bfloat16)
        out = layer.tree(x, parents)
        layer.accept(torch.cat([x[paths[0]], x[6:][paths[1]]]), [3, 3])
        print(f"step {i}: trees of 6 and 4 nodes, norm {float(out.float().norm()):.2f}; lengths {layer.lens.tolist()}")


if __name__ == "__main__":
    main()
