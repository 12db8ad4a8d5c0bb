"""Latent, expanded and tree attention beside and behind one another: on streams of their own at once, and after calls
that leave other things in the SMs' shared memory."""
import pytest
import torch

import kda_decode_recurrence_gb300 as kda

from _latent import HEAD, LATENT, ROPE, ROW, LatentCase, mask_of, trees
from _paged import Case, cumulative

pytestmark = pytest.mark.gpu


def normal(seed, *shape, amplitude=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * amplitude).to(torch.bfloat16).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Latent:
    def __init__(self, n, lens, H, page, amplitude=1.0, tree=False):
        self.c, self.q = LatentCase(n, lens, page, seed=91), normal(92, sum(n), H, ROW, amplitude=amplitude)
        self.mask = mask_of(trees(n), -(-max(n) // 32)) if tree else None
        self.shape = (sum(n), H, LATENT)

    def run(self, out, lse, **kw):
        c = self.c
        return kda.kda_latent_attention(out, self.q, c.cache, c.cu, c.seq_lens, c.table, tree_mask=self.mask, lse=lse, **kw)


class Expanded:
    def __init__(self, n, lens, H, amplitude=1.0):
        self.q, self.kv = normal(93, sum(n), H, HEAD + ROPE, amplitude=amplitude), normal(94, sum(lens), H, 2 * HEAD)
        self.pe, self.cu, self.shape = normal(95, sum(lens), ROPE), (ints(cumulative(n)), ints(cumulative(lens))), (sum(n), H, HEAD)

    def run(self, out, lse, **kw):
        return kda.kda_latent_expanded(out, self.q, self.kv, self.pe, *self.cu, lse=lse, **kw)


class Tree:
    def __init__(self, n, lens, H, HKV, D, cache, amplitude=1.0):
        self.c, self.q = Case(n, lens, HKV, D, 64, cache=cache, seed=96), normal(97, sum(n), H, D, amplitude=amplitude)
        self.mask, self.most, self.shape = mask_of(trees(n), -(-max(n) // 32)), max(n), (sum(n), H, D)

    def run(self, out, lse, **kw):
        caches, scales = self.c.args()
        return kda.kda_tree_attention(out, self.q, *caches, self.c.cu, self.c.seq_lens, self.c.table, self.mask, self.most,
                                      lse=lse, **scales, **kw)


def outputs(call):
    return torch.zeros(call.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(call.shape[:2], device="cuda")


def alone(call):
    out, lse = outputs(call)
    assert int(call.run(out, lse).item()) == 0
    return out, lse


def test_at_once_on_many_streams():
    calls = [Latent([1] * 40, [300 + 97 * i for i in range(40)], 32, 64), Expanded([300, 129, 40], [900, 129, 700], 6),
             Tree([40, 13, 60], [2000, 530, 900], 12, 2, 128, "bf16"), Latent([5, 40], [1500, 130], 24, 16, tree=True),
             Tree([40, 13, 60], [2000, 530, 900], 24, 2, 128, "e4m3"), Tree([40, 13], [2000, 530], 8, 2, 64, "e4m3")]
    want = [alone(c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    for turn in range(6):
        got = [outputs(c) for c in calls]
        torch.cuda.synchronize()
        words = [c.run(*o, stream=s) for _ in range(4) for c, o, s in zip(calls, got, streams)]
        torch.cuda.synchronize()
        assert all(int(w.item()) == 0 for w in words)
        for (out, lse), (o, e) in zip(got, want):
            assert torch.equal(out, o) and torch.equal(lse, e), f"turn {turn}"


@pytest.mark.parametrize("make", [lambda a: Latent([5] * 20, [700 + 31 * i for i in range(20)], 24, 64, a),
                                  lambda a: Expanded([250, 129, 1], [600, 300, 40], 5, a)], ids=["latent", "expanded"])
def test_bits_do_not_depend_on_what_ran_before(make):
    """Row tiles that are not full: what the other rows hold is left over from the calls before."""
    call = make(1.0)
    want = alone(call)
    full = [lambda a: Latent([1] * 152, [1100] * 152, 128, 64, a), lambda a: Expanded([512] * 8, [512] * 8, 8, a),
            lambda a: Tree([64] * 20, [1100] * 20, 32, 8, 128, "bf16", a)]
    for before in full:
        for amplitude in (1e-3, 30.0, 1e3):
            alone(before(amplitude))
            out, lse = alone(call)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), f"after queries of {amplitude}"
