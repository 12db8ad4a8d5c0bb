"""The latent layer of examples/latent_tree_step.py: prompts, trees and accepted paths in a row, against the
formula in 64 bits on the cached rows, and each node against its path alone."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import latent_tree_step as ex  # noqa: E402

from _latent import softmax64  # noqa: E402
from _paged import U_BF16  # noqa: E402

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def heads64(layer, q, rows, see):
    """(outputs, tolerances) [n, H, 128] of queries q [n, H, 192] over cached rows [L, 576], in 64 bits.

    Beside softmax64's tolerance: keys and values (expanded form) or queries and sums (absorbed form) are rounded
    to bf16 once more.  A key's entries are each off by U: its score by U scale sum |q||k| at most; a query
    absorbed into the latents likewise by U scale sum |q~||c|.  That moves each weight by twice that,
    once in the sum too.  A value or a sum rounded to bf16 moves an output by U of what it adds up in magnitude.
    The matrix products themselves add 512 or 128 fp32 roundings, less than U / 64 of the same sums."""
    c, pe = rows[:, :512].double(), rows[:, 512:].double()
    k = torch.cat([torch.einsum("lc,hcd->lhd", c, layer.w_k.double()), pe[:, None].expand(-1, ex.HEADS, -1)], -1)
    v = torch.einsum("lc,hcd->lhd", c, layer.w_v.double())
    out, _, tol, _ = softmax64(q, k, v, see, SCALE)
    absorbed = torch.cat([torch.einsum("nhd,hcd->nhc", q[..., :128].double(), layer.w_k.double()), q[..., 128:].double()], -1)
    for h in range(ex.HEADS):
        direct = SCALE * (q[:, h].double().abs() @ k[:, h].abs().T)
        via = SCALE * (absorbed[:, h].abs() @ rows.double().abs().T)
        off = 1.02 * U_BF16 * torch.where(see, torch.maximum(direct, via), 0.0).amax(1)
        x = torch.where(see, SCALE * (q[:, h].double() @ k[:, h].T), -torch.inf)
        P = torch.softmax(x, 1)
        mass = P @ v[:, h].abs()                                     # of values rounded one by one
        sums = P @ c                                                  # of the latents' sum, rounded, then projected
        spread = (P @ c.abs()) @ layer.w_v[h].double().abs()
        tol[:, h] += 2 * off[:, None] * mass + 1.02 * U_BF16 * (mass + sums.abs() @ layer.w_v[h].double().abs())
        tol[:, h] += (U_BF16 + 2 * off[:, None]) * spread            # weights rounded, in the absorbed form before w_v
    return out, tol


def near(out, want):
    off = (out.double() - want[0]).abs()
    assert bool((off <= want[1]).all()), f"off by {float((off / want[1]).max()):.3g} tolerances"


def test_prompt_then_trees_then_accepted_paths():
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda n: torch.randn(n, ex.DIM, device="cuda", generator=g).to(torch.bfloat16)
    layer, n = ex.Layer(2, pages_each=12), [37, 20]
    x = rand(sum(n))
    out = layer.prompt(x, n)
    at = 0
    for b, k in enumerate(n):
        q, _ = layer.project(x[at:at + k], torch.arange(k, device="cuda"))
        see = torch.ones(k, k, dtype=torch.bool, device="cuda").tril()
        near(out[at:at + k], heads64(layer, q, layer.rows_of(b, k), see))
        at += k
    parents = [[-1, 0, 0, 1, 1, 2, 3], [-1, -1, 0, 2]]
    paths = [[0, 1, 4], [0, 2, 3]]
    for _ in range(3):
        x = rand(11)
        lens = layer.lens.tolist()
        out = layer.tree(x, parents)
        t = 0
        for b, p in enumerate(parents):
            rows = layer.rows_of(b, lens[b] + len(p))
            see = torch.zeros(len(p), lens[b] + len(p), dtype=torch.bool)
            see[:, :lens[b]] = True
            depth = []
            for i, parent in enumerate(p):
                if parent >= 0:
                    see[i] |= see[parent]
                see[i, lens[b] + i] = True
                depth.append(depth[parent] + 1 if parent >= 0 else 0)
            q, _ = layer.project(x[t:t + len(p)], torch.tensor(depth, device="cuda") + lens[b])
            near(out[t:t + len(p)], heads64(layer, q, rows, see.cuda()))
            t += len(p)
        # an accepted path's rows, appended one behind the other, are those that its nodes had
        nodes = [layer.rows_of(b, lens[b] + len(p))[lens[b]:].clone() for b, p in enumerate(parents)]
        layer.accept(torch.cat([x[paths[0]], x[7:][paths[1]]]), [3, 3])
        assert layer.lens.tolist() == [k + 3 for k in lens]
        for b in range(2):
            rows = layer.rows_of(b, lens[b] + 3)[lens[b]:].float()
            # (rows of another batch's matrix product may round otherwise: a step of bf16)
            assert bool(((rows - nodes[b][paths[b]].float()).abs() <= 4 * U_BF16 * rows.abs().clamp_min(2.0 ** -6)).all())


def test_a_node_is_as_its_path_alone():
    """Each leaf's path as a tree of its own (a chain): the same outputs, within the roundings of a product with
    other shapes."""
    g = torch.Generator(device="cuda").manual_seed(6)
    layer, n = ex.Layer(1, pages_each=12), [30]
    layer.prompt(torch.randn(30, ex.DIM, device="cuda", generator=g).to(torch.bfloat16), n)
    parents = [-1, 0, 0, 1, 2, 4]
    x = torch.randn(6, ex.DIM, device="cuda", generator=g).to(torch.bfloat16)
    out = layer.tree(x, [parents])
    rows = layer.rows_of(0, 36)
    for path in ([0, 1, 3], [0, 2, 4, 5]):
        alone = layer.tree(x[path], [list(range(-1, len(path) - 1))])
        q, _ = layer.project(x[path], torch.arange(30, 30 + len(path), device="cuda"))
        see = torch.ones(len(path), 30 + len(path), dtype=torch.bool, device="cuda").tril(30)
        want = heads64(layer, q, torch.cat([rows[:30], rows[30:][path]]), see)
        near(out[path], want)
        near(alone, want)


def test_main_runs(capsys):
    ex.main()
    assert "lengths" in capsys.readouterr().out
