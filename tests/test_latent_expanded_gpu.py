"""kda_latent_expanded against softmax attention in 64 bits (tolerances: see _latent.softmax64)."""
import pytest
import torch

import kda_decode_recurrence_gb300 as kda

from _latent import HEAD, ROPE, SCALE, close, seen_by, softmax64
from _paged import cumulative
from _parity import Guarded

pytestmark = pytest.mark.gpu


class Prompts:
    """Tokens, keys and values of requests on the device: q and kv strided by one head more, k_pe the last
    columns of wider rows."""

    def __init__(self, n, lens, H, seed=0, amplitude=1.0, tail=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.lens, self.H = list(n), list(lens), H
        Tq, Tk = sum(n), sum(lens) + tail
        make = lambda *s: (torch.randn(*s, generator=g) * amplitude).to(torch.bfloat16).cuda()
        self.q = make(Tq, H + 1, HEAD + ROPE)[:, :H]
        self.kv = make(Tk, H + 1, 2 * HEAD)[:, :H]
        self.k_pe = make(Tk, 3 * ROPE)[:, 2 * ROPE:]
        self.cu_q = torch.tensor(cumulative(self.n), dtype=torch.int32, device="cuda")
        self.cu_k = torch.tensor(cumulative(self.lens), dtype=torch.int32, device="cuda")


def attend(c, causal=True, scale=None, with_lse=True, **kw):
    T, H = c.q.shape[:2]
    out = Guarded((T, H, HEAD), torch.bfloat16, fill=float("nan"))
    lse = Guarded((T, H), torch.float32, fill=float("nan"))
    work = Guarded((kda.latent_expanded_workspace_size(len(c.n), T, H),), torch.uint8, fill=0xFF)
    status = kda.kda_latent_expanded(out.t, c.q, c.kv, c.k_pe, c.cu_q, c.cu_k, scale=scale, causal=causal,
                                     lse=lse.t if with_lse else None, workspace=work.t, **kw)
    torch.cuda.synchronize()
    assert out.intact() and lse.intact() and work.intact()
    return out.t, lse.t, int(status.item())


def reference(c, causal=True, scale=SCALE):
    parts, cq, ck = [], cumulative(c.n), cumulative(c.lens)
    for b in range(len(c.n)):
        at = slice(ck[b], ck[b + 1])
        kv = c.kv[at].double()
        k = torch.cat([kv[..., :HEAD], c.k_pe[at].double()[:, None].expand(-1, c.H, -1)], -1)
        parts.append(softmax64(c.q[cq[b]:cq[b + 1]], k, kv[..., HEAD:], seen_by(c.n[b], c.lens[b], causal), scale))
    return [torch.cat(x) for x in zip(*parts)]


def check(c, causal=True, scale=None, **kw):
    out, lse, status = attend(c, causal, scale, **kw)
    assert status == 0
    close(out, lse, reference(c, causal, SCALE if scale is None else scale))
    return out, lse


SHAPES = [
    dict(n=[1], lens=[1], H=1),
    dict(n=[1, 1, 1], lens=[127, 128, 129], H=3),
    dict(n=[7], lens=[300], H=16),
    dict(n=[128], lens=[128], H=4),
    dict(n=[129, 64, 1], lens=[129, 200, 640], H=5),
    dict(n=[0, 30, 0, 255], lens=[0, 30, 12, 300], H=8),
    dict(n=[256, 257], lens=[256, 257], H=2),
    dict(n=[5, 9], lens=[3, 0], H=4),                       # padding: more tokens than keys
    dict(n=[600], lens=[1411], H=3),
    dict(n=[33, 700, 290], lens=[33, 700, 290], H=12),
    dict(n=[1500], lens=[1500], H=1),
]
IDS = [f"n{max(s['n'])}_L{max(s['lens'])}_H{s['H']}" for s in SHAPES]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_shapes(shape, causal):
    check(Prompts(**shape), causal)
