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
    if "stream" in kw:  # (the buffers are filled on the current one)
        kw["stream"].wait_stream(torch.cuda.current_stream())
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


@pytest.mark.parametrize("amplitude,scale", [(1.0, 3.0), (30.0, 1.0), (1e4, 1.0), (1.0, -0.3), (1.0, 0.0)])
def test_scores_of_other_sizes(amplitude, scale):
    c = Prompts([100, 300], [220, 300], 3, seed=61)
    c.q.mul_(amplitude)
    check(c, scale=scale)


@pytest.mark.parametrize("amplitude", [2.0 ** -110, 2.0 ** 110])
def test_values_of_extreme_size(amplitude):
    c = Prompts([100, 300], [220, 300], 3, seed=62)
    c.kv[..., HEAD:] *= amplitude
    check(c)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n,L", [(5, 70), (90, 300), (300, 300), (600, 600)])
def test_a_bad_value_reaches_only_the_tokens_that_see_it(n, L, bad):
    """A later token's V that is not finite, in either half of the columns; a neighbour request is as before."""
    for col in (5, 100):
        c = Prompts([n, 40], [L, 90], 2, seed=63)
        want, wlse, _ = attend(c)
        i = (2 * n) // 3
        c.kv[L - n + i, 1, HEAD + col] = bad
        out, lse, status = attend(c)
        assert status == 0 and torch.equal(lse, wlse)
        assert torch.equal(out[:i], want[:i]) and torch.equal(out[n:], want[n:]) and torch.equal(out[:, 0], want[:, 0])
        keep = torch.arange(HEAD, device="cuda") != col
        assert torch.equal(out[i:n, 1][:, keep], want[i:n, 1][:, keep])
        assert not bool(torch.isfinite(out[i:n, 1, col]).any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_key_reaches_only_the_tokens_that_see_it(bad):
    c = Prompts([200, 40], [300, 90], 2, seed=64)
    want, wlse, _ = attend(c)
    c.k_pe[240] = float("nan")                     # token 140's position part: all heads
    c.kv[350:390] = bad                            # the second request's last 40 keys and values: its own tokens'
    out, lse, status = attend(c)
    assert status == 0 and torch.equal(out[:140], want[:140]) and torch.equal(lse[:140], wlse[:140])
    assert bool(torch.isnan(out[140:200]).all())
    # what lies behind a request's keys is the next one's
    c = Prompts([200], [300], 2, seed=64, tail=100)
    want, wlse, _ = attend(Prompts([200], [300], 2, seed=64, tail=100))
    c.kv[300:] = bad
    c.k_pe[300:] = bad
    cu = c.cu_k.clone()
    out, lse, status = attend(c)
    assert status == kda.DEV_BAD_SEQLEN and torch.equal(cu, c.cu_k)         # (cu_k does not span the 400 keys)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_no_keys_at_all():
    c = Prompts([3, 2], [0, 0], 4, seed=65)
    check(c)


def test_without_lse_and_on_another_stream():
    c = Prompts([33, 300], [50, 700], 5, seed=66)
    want, _, _ = attend(c)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out, _, status = attend(c, with_lse=False, stream=stream)
    assert status == 0 and torch.equal(out, want)


def test_same_bits_and_graph_replay():
    c = Prompts([300, 40, 129], [700, 40, 300], 5, seed=67)
    want, wlse, _ = attend(c)
    again, alse, _ = attend(c)
    assert torch.equal(want, again) and torch.equal(wlse, alse)
    other = torch.tensor(cumulative([500, 240, 300]), dtype=torch.int32, device="cuda")
    long = c.cu_k.clone()
    c.cu_k.copy_(other)
    less, llse, _ = attend(c)
    out, lse = torch.zeros_like(want), torch.zeros_like(wlse)
    work = torch.empty(kda.latent_expanded_workspace_size(3, 469, 5), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_latent_expanded(out, c.q, c.kv, c.k_pe, c.cu_q, c.cu_k, lse=lse, workspace=work, dev_status=status)
    for now, (o, e) in ((other, (less, llse)), (long, (want, wlse)), (other, (less, llse))):
        c.cu_k.copy_(now)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, e) and int(status.item()) == 0


def test_same_bits_when_copies_arrive_late():
    c = Prompts([1100, 700], [6000, 5000], 8, seed=68)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    first = None
    for trial in range(8):
        if trial % 2 == 0:
            flush.fill_(trial)
        out, lse, status = attend(c)
        first = first or (out, lse)
        assert status == 0 and torch.equal(out, first[0]) and torch.equal(lse, first[1]), f"trial {trial}"


def test_bad_offsets_are_reported_and_skipped():
    """(The others are served, not with the same bits: the call is cut elsewhere.)"""
    c = Prompts([9, 40, 2], [90, 140, 30], 4, seed=69)
    want = reference(c)

    def served(out, lse, rows):
        close(out[rows], lse[rows], [x[rows] for x in want])

    for name, bad in (("cu_k", [0, 90, 20, 260]), ("cu_q", [0, 9, 8, 51])):      # the second ends before it begins
        keep = getattr(c, name).clone()
        getattr(c, name).copy_(torch.tensor(bad, dtype=torch.int32))
        out, lse, status = attend(c)
        assert status == kda.DEV_BAD_SEQLEN
        served(out, lse, slice(0, 9 if name == "cu_k" else 8))
        getattr(c, name).copy_(keep)
    c.cu_q.copy_(torch.tensor([0, 9, 49, 49], dtype=torch.int32))                # the last two rows are nobody's
    out, lse, status = attend(c)
    assert status == kda.DEV_BAD_SEQLEN and bool(torch.isnan(out[49:]).all())
    served(out, lse, slice(0, 49))


def test_offsets_beyond_32_bits():
    """Keys past 2^31 elements of kv, behind those of a request without new tokens."""
    n, L, far, H = 130, 300, 90000, 100
    g = torch.Generator(device="cuda").manual_seed(70)
    kv = torch.zeros(far + L, H, 2 * HEAD, device="cuda", dtype=torch.bfloat16)
    kv[far:] = torch.randn(L, H, 2 * HEAD, device="cuda", generator=g)
    pe = torch.randn(far + L, ROPE, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(n, H, HEAD + ROPE, device="cuda", generator=g).to(torch.bfloat16)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out, want = torch.empty(2, n, H, HEAD, device="cuda", dtype=torch.bfloat16).unbind()
    kda.kda_latent_expanded(out, q, kv, pe, ints([0, 0, n]), ints([0, far, far + L]), check_device=True)
    kda.kda_latent_expanded(want, q, kv[far:], pe[far:], ints([0, n]), ints([0, L]), check_device=True)
    assert torch.equal(out, want)


def test_many_requests():
    g = torch.Generator().manual_seed(71)
    lens = torch.randint(0, 40, (800,), generator=g).tolist()
    check(Prompts([min(x, i % 3) for i, x in enumerate(lens)], lens, 2, seed=71))


def test_one_long_prompt_in_many_pieces():
    check(Prompts([700], [9000], 1, seed=72))


@pytest.mark.parametrize("causal", [True, False])
def test_queries_of_padding_tokens_have_no_influence(causal):
    """Tokens before position 0 hold anything: huge numbers, infinities, NaN.  Their rows stand in the same warps as those of
    tokens that see something."""
    c = Prompts([50, 9, 300], [33, 0, 290], 3, seed=73)
    want, wlse, _ = attend(c, causal)
    at = cumulative(c.n)
    for junk in (3e38, float("inf"), float("nan")):
        for b in range(3):
            c.q[at[b]:at[b] + max(0, c.n[b] - c.lens[b])] = junk
        out, lse, status = attend(c, causal)
        assert status == 0 and torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_key_of_the_second_request(bad):
    """Keys and values that its later tokens see: the earlier ones, and the first request, keep their bits."""
    c = Prompts([200, 140], [300, 490], 2, seed=74)
    want, wlse, _ = attend(c)
    c.kv[700:710, 1] = bad                          # positions 400 .. 409: the second request's tokens from 50 on
    out, lse, status = attend(c)
    assert status == 0 and torch.equal(out[:250], want[:250]) and torch.equal(lse[:250], wlse[:250])
    assert torch.equal(out[:, 0], want[:, 0]) and torch.equal(lse[:, 0], wlse[:, 0])
    if bad != bad:
        assert bool(torch.isnan(out[250:, 1]).all()) and bool(torch.isnan(lse[250:, 1]).all())
    else:                                           # (scores of -infinity leave their own values' columns only)
        assert not bool(torch.isfinite(out[250:, 1]).any())
