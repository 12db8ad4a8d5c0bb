"""kda_latent_attention against softmax attention in 64 bits (tolerances: see _latent.softmax64).
Rows of the cache that no position in use owns hold NaN throughout."""
import pytest
import torch

import kda_decode_recurrence_gb300 as kda

from _latent import LATENT, ROW, SCALE, LatentCase, close, mask_of, seen_by, softmax64, trees
from _paged import cumulative
from _parity import Guarded

pytestmark = pytest.mark.gpu


def queries(case, H, seed=1, amplitude=1.0):
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn(case.T, H + 1, ROW, generator=g) * amplitude).to(torch.bfloat16).cuda()
    return wide[:, :H]                      # tokens strided by (H + 1) 576


def attend(case, q, causal=True, mask=None, scale=None, with_lse=True, **kw):
    """The call on guarded outputs and workspace; returns (out, lse, status)."""
    T, H, _ = q.shape
    out = Guarded((T, H, LATENT), torch.bfloat16, fill=float("nan"))
    lse = Guarded((T, H), torch.float32, fill=float("nan"))
    work = Guarded((kda.latent_attention_workspace_size(case.B, T, H),), torch.uint8, fill=0xFF)
    status = kda.kda_latent_attention(out.t, q, kw.pop("cache", case.cache), kw.pop("cu", case.cu),
                                      kw.pop("seq_lens", case.seq_lens), kw.pop("table", case.table), scale=scale,
                                      causal=causal, tree_mask=mask, lse=lse.t if with_lse else None, workspace=work.t, **kw)
    torch.cuda.synchronize()
    assert out.intact() and lse.intact() and work.intact()
    return out.t, lse.t, int(status.item())


def reference(case, q, causal=True, tree=None, scale=SCALE, table=None):
    parts = []
    cu = cumulative(case.n)
    for b in range(case.B):
        rows = case.dense(b, table)
        see = seen_by(case.n[b], max(case.lens[b], 0), causal, tree[b] if tree else None)
        parts.append(softmax64(q[cu[b]:cu[b + 1]], rows[:, None], rows[:, None, :LATENT], see, scale))
    return [torch.cat(x) for x in zip(*parts)]


def check(case, q, causal=True, tree=None, scale=None, table=None, words=None, **kw):
    mask = None if tree is None else mask_of(tree, words or -(-max(max(case.n), 1) // 32))
    if table is not None:
        kw["table"] = table
    out, lse, status = attend(case, q, causal, mask, scale, **kw)
    assert status == 0
    close(out, lse, reference(case, q, causal, tree, SCALE if scale is None else scale, table))
    return out, lse


SHAPES = [
    # single tokens: one position, page and tile edges, few and many heads
    dict(n=[1], lens=[1], H=1, page=16),
    dict(n=[1], lens=[517], H=16, page=64),
    dict(n=[1] * 7, lens=[1, 63, 64, 65, 127, 128, 129], H=8, page=16),
    dict(n=[1] * 5, lens=[255, 256, 257, 300, 33], H=96, page=128),
    dict(n=[1, 1, 1], lens=[700, 2, 1025], H=128, page=32),
    dict(n=[1], lens=[12000], H=12, page=64),
    dict(n=[1] * 3, lens=[1100, 128, 640], H=130, page=64),
    # windows, empty requests, padding (more new tokens than positions)
    dict(n=[1, 2, 3, 4, 5, 6, 7, 8], lens=[9, 2, 100, 64, 130, 6, 65, 257], H=8, page=16),
    dict(n=[0, 5, 0, 3], lens=[0, 40, 12, 3], H=5, page=16),
    dict(n=[4, 6, 3], lens=[2, 0, 50], H=40, page=16),
    dict(n=[8, 8], lens=[520, 41], H=64, page=32),
    # rows of many tiles, with and without a cached prefix
    dict(n=[40], lens=[40], H=64, page=16),
    dict(n=[33, 1, 0, 20], lens=[230, 900, 5, 300], H=24, page=64),
    dict(n=[130], lens=[390], H=128, page=64),
]
IDS = [f"n{max(s['n'])}_L{max(s['lens'])}_H{s['H']}_p{s['page']}" for s in SHAPES]


def make(shape, **kw):
    shape = dict(shape)
    H = shape.pop("H")
    case = LatentCase(**shape, **kw)
    return case, queries(case, H)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_shapes(shape, causal):
    case, q = make(shape)
    check(case, q, causal)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_trees(shape):
    case, q = make(shape)
    check(case, q, tree=trees(case.n, seed=5))
