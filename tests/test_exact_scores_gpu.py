"""The attention calls on scores that fp32 holds exactly: queries and keys of small whole numbers, the
queries times powers of two up to 2^60.

A score is then a whole number S (below 2^14 in size) times 2^e, and the tolerances need no term of the scores'
sums, which elsewhere grows with the scores until it hides everything:
  - x = S 2^e log2 e is rounded, and so is the maximum m: each by half an fp32 step of |x|, the factor log2 e
    likewise, so that a weight is off by 4 U |x|, and by the exponential's 2^-21;
  - from 2^e = 2^10 on two different scores are 1000 and more apart: the weights of all but the largest are 0 in
    fp32, and the largest, being equal, stay equal whatever their rounding.  out is the mean of their values.
  - a weight is e^(x - m), at most 1, with an fp32 exponent: below 2^-126 it is 0, and the row's sum of weights is
    at least 1, so that L of them move the output by L 2^-126 of the largest value.
Beyond that the weights' and outputs' rounding to bf16 and the fp32 sums count, as in _latent.softmax64."""
import math

import pytest
import torch

import kda_decode_recurrence_gb300 as kda

from _latent import HEAD, LATENT, ROPE, ROW, LatentCase, close, mask_of, seen_by, trees
from _paged import Case, U_BF16, U_F32, cumulative

pytestmark = pytest.mark.gpu

# Powers of two of the queries, dealt to the tokens in turn.
SPREADS = {"small": [0], "past_the_rounding": [14, 15, 16, 17, 18], "billions": [24, 31, 40, 60], "mixed": [0, 40, 3, 0, 17, 60, 1]}


def whole(g, *shape, most=3):
    return torch.randint(-most, most + 1, shape, generator=g).float()


def powers(T, spread):
    return torch.tensor([SPREADS[spread][t % len(SPREADS[spread])] for t in range(T)])


def times_powers(q, e):
    return (q * torch.exp2(e.float())[:, None, None]).to(torch.bfloat16)


def exact64(q, e, k, v, see):
    """(out, lse, tolerances) of whole queries q [n, H, Dk], times 2^e [n] and scale 1."""
    n, H, _ = q.shape
    L, Dv = v.shape[0], v.shape[2]
    out = torch.zeros(n, H, Dv, dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    if L == 0 or n == 0:
        return out, lse, tol, ltol
    some, size, count = see.any(1), torch.exp2(e.double())[:, None], see.sum(1).double()
    for h in range(H):
        kk, vv = k[:, min(h, k.shape[1] - 1)].double(), v[:, min(h, v.shape[1] - 1)].double()
        s = q[:, h].double() @ kk.T
        assert float(s.abs().max()) < 2 ** 14
        x = torch.where(see, s * size, -math.inf)
        top = torch.where(some, x.amax(1), 0.0)
        w = torch.exp(x - top[:, None])
        total = torch.where(some, w.sum(1), 1.0)
        P = w / total[:, None]
        o, mass = P @ vv, P @ vv.abs()
        largest = torch.where(see, x.abs(), 0.0).amax(1)
        off = torch.where(e.to(q.device) >= 10, 0.0, 4 * U_F32 * 1.4427 * largest) + 2.0 ** -21
        out[:, h], lse[:, h] = o, torch.where(some, top + torch.log(total), -math.inf)
        tol[:, h] = (U_BF16 + 2 * off + count * U_F32)[:, None] * mass + U_BF16 * o.abs() + L * 2.0 ** -126 * vv.abs().amax()
        ltol[:, h] = torch.where(some, off + (count + 1) * U_F32 + largest * 8 * U_F32, 0.0)
    assert float((tol.median() / out.abs().mean())) < 0.05  # (a tolerance that hides the values says nothing)
    return out, lse, tol, ltol


def joined(parts):
    return [torch.cat(x) for x in zip(*parts)]


@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("n,lens,H", [([1], [1], 3), ([1, 1, 1], [200, 3000, 129], 16), ([7, 40], [9000, 130], 24),
                                      ([130], [390], 8), ([1] * 60, [100 + 31 * i for i in range(60)], 5)])
def test_latent(n, lens, H, spread):
    for kind in ("causal", "full", "tree"):
        case = LatentCase(n, lens, 16, seed=81)
        g = torch.Generator().manual_seed(82)
        used = case.used.cuda()
        case.cache[used] = whole(g, *case.cache.shape, most=1).to(torch.bfloat16).cuda()[used]
        q, e = whole(g, case.T, H, ROW, most=2), powers(case.T, spread)
        tree = trees(case.n, seed=4) if kind == "tree" else None
        out, lse = torch.empty(case.T, H, LATENT, dtype=torch.bfloat16, device="cuda"), torch.empty(case.T, H, device="cuda")
        status = kda.kda_latent_attention(out, times_powers(q, e).cuda(), case.cache, case.cu, case.seq_lens, case.table, scale=1.0,
                                          causal=kind == "causal", tree_mask=mask_of(tree, -(-max(n) // 32)) if tree else None, lse=lse)
        assert int(status.item()) == 0
        parts, cu, q = [], cumulative(n), q.cuda()
        for b in range(case.B):
            rows, at = case.dense(b), slice(cu[b], cu[b + 1])
            see = seen_by(n[b], lens[b], kind == "causal", tree[b] if tree else None)
            parts.append(exact64(q[at], e[at].cuda(), rows[:, None], rows[:, None, :LATENT], see))
        close(out, lse, joined(parts))


@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("n,lens,H", [([1], [1], 3), ([30, 1, 300], [200, 3000, 300], 4), ([700], [9000], 1),
                                      ([33 + 7 * i for i in range(20)], [200 + 31 * i for i in range(20)], 6)])
def test_expanded(n, lens, H, spread):
    g = torch.Generator().manual_seed(83)
    Tq, Tk = sum(n), sum(lens)
    q, e = whole(g, Tq, H, HEAD + ROPE, most=2), powers(Tq, spread)
    kv, pe = (whole(g, *s).to(torch.bfloat16).cuda() for s in ((Tk, H, 2 * HEAD), (Tk, ROPE)))
    ints = lambda x: torch.tensor(cumulative(x), dtype=torch.int32, device="cuda")
    for causal in (True, False):
        out, lse = torch.empty(Tq, H, HEAD, dtype=torch.bfloat16, device="cuda"), torch.empty(Tq, H, device="cuda")
        status = kda.kda_latent_expanded(out, times_powers(q, e).cuda(), kv, pe, ints(n), ints(lens), scale=1.0, causal=causal, lse=lse)
        assert int(status.item()) == 0
        parts, cq, ck, whole_q = [], cumulative(n), cumulative(lens), q.cuda()
        for b in range(len(n)):
            at, to = slice(ck[b], ck[b + 1]), slice(cq[b], cq[b + 1])
            k = torch.cat([kv[at, :, :HEAD], pe[at][:, None].expand(-1, H, -1)], -1)
            parts.append(exact64(whole_q[to], e[to].cuda(), k, kv[at, :, HEAD:], seen_by(n[b], lens[b], causal)))
        close(out, lse, joined(parts))


@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,lens,H,HKV", [([1], [1], 1, 1), ([13, 40], [517, 300], 12, 2), ([11, 3], [9000, 200], 8, 2),
                                          ([1 + i % 30 for i in range(40)], [60 + 17 * i for i in range(40)], 6, 2)])
def test_tree(n, lens, H, HKV, D, cache, spread):
    case = Case(n, lens, HKV, D, 16, cache=cache, seed=84)
    g = torch.Generator().manual_seed(85)
    used = case.used.cuda()
    for x, s in case.tensors.values():
        y = whole(g, *x.shape).cuda()
        if s is None:
            x[used] = y.to(torch.bfloat16)[used]
        else:  # codes of whole numbers, scales of 1, 2 and 4
            x.view(torch.uint8)[used] = y.to(torch.float8_e4m3fn).view(torch.uint8)[used]
            s[used] = torch.exp2(torch.randint(0, 3, s.shape, generator=g).float()).cuda()[used]
    tree, q, e = trees(n, seed=4), whole(g, case.T, H, D, most=2), powers(case.T, spread)
    caches, scales = case.args()
    out, lse = torch.empty(case.T, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(case.T, H, device="cuda")
    status = kda.kda_tree_attention(out, times_powers(q, e).cuda(), *caches, case.cu, case.seq_lens, case.table, mask_of(tree, -(-max(n) // 32)),
                                    max(n), scale=1.0, **scales, lse=lse)
    assert int(status.item()) == 0
    parts, cu, G, q = [], cumulative(n), H // HKV, q.cuda()
    for b in range(case.B):
        k, v = (case.dense(x, b).repeat_interleave(G, 1) for x in "kv")
        at = slice(cu[b], cu[b + 1])
        parts.append(exact64(q[at], e[at].cuda(), k, v, seen_by(n[b], lens[b], nodes=tree[b])))
    close(out, lse, joined(parts))
