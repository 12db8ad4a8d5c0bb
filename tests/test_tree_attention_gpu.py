"""kda_tree_attention against softmax attention in 64 bits under each node's mask (tolerances: see
_latent.softmax64).  Rows of the cache that no position in use owns hold NaN throughout."""
import pytest
import torch

import kda_decode_recurrence_gb300 as kda

from _latent import close, mask_of, seen_by, softmax64, trees
from _paged import Case, cumulative
from _parity import Guarded

pytestmark = pytest.mark.gpu


def queries(case, H, seed=1, amplitude=1.0):
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn(case.T, H + 2, case.D, generator=g) * amplitude).to(torch.bfloat16).cuda()
    return wide[:, :H]


def attend(case, q, mask, scale=None, max_tokens=None, with_lse=True, **kw):
    T, H, D = q.shape
    out = Guarded((T, H, D), torch.bfloat16, fill=float("nan"))
    lse = Guarded((T, H), torch.float32, fill=float("nan"))
    most = max(case.n) if max_tokens is None else max_tokens
    work = Guarded((kda.tree_attention_workspace_size(case.B, T, most, H, case.HKV, D),), torch.uint8, fill=0xFF)
    caches, scales = case.args()
    status = kda.kda_tree_attention(out.t, q, *caches, kw.pop("cu", case.cu), kw.pop("seq_lens", case.seq_lens),
                                    kw.pop("table", case.table), mask, most, scale=scale, **scales,
                                    lse=lse.t if with_lse else None, workspace=work.t, **kw)
    torch.cuda.synchronize()
    assert out.intact() and lse.intact() and work.intact()
    return out.t, lse.t, int(status.item())


def reference(case, q, tree, scale, table=None):
    G, cu, parts = q.shape[1] // case.HKV, cumulative(case.n), []
    for b in range(case.B):
        k, v = (case.dense(x, b, table).repeat_interleave(G, 1) for x in ("k", "v"))
        see = seen_by(case.n[b], max(case.lens[b], 0), nodes=tree[b])
        parts.append(softmax64(q[cu[b]:cu[b + 1]], k, v, see, scale))
    return [torch.cat(x) for x in zip(*parts)]


def check(case, q, tree, scale=None, words=None, table=None, **kw):
    mask = mask_of(tree, words or -(-max(max(case.n), 1) // 32))
    if table is not None:
        kw["table"] = table
    out, lse, status = attend(case, q, mask, scale, **kw)
    assert status == 0
    close(out, lse, reference(case, q, tree, q.shape[2] ** -0.5 if scale is None else scale, table))
    return out, lse


SHAPES = [
    dict(n=[1], lens=[1], H=1, HKV=1, D=128, page=16),
    dict(n=[13], lens=[530], H=32, HKV=8, D=128, page=64),
    dict(n=[1, 2, 3, 9, 17], lens=[1, 130, 64, 129, 300], H=8, HKV=2, D=64, page=16),
    dict(n=[33, 64, 20], lens=[161, 128, 20], H=4, HKV=2, D=128, page=16),
    dict(n=[65, 0, 40], lens=[70, 3, 600], H=12, HKV=1, D=128, page=128),
    dict(n=[4, 6, 3], lens=[2, 0, 50], H=4, HKV=2, D=128, page=16),      # padding
    dict(n=[200], lens=[290], H=3, HKV=1, D=64, page=32),
    dict(n=[30, 12], lens=[2000, 45], H=20, HKV=2, D=128, page=64),
    dict(n=[5], lens=[3000], H=128, HKV=1, D=128, page=64),
]
IDS = [f"n{max(s['n'])}_L{max(s['lens'])}_H{s['H']}_{s['HKV']}_D{s['D']}_p{s['page']}" for s in SHAPES]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_shapes(shape, cache):
    shape = dict(shape)
    H = shape.pop("H")
    case = Case(**shape, cache=cache)
    check(case, queries(case, H), trees(case.n, seed=7))
