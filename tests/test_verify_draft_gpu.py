"""kda_verify_draft against the definition with exact sums: tokens and counts are equal."""
import numpy as np
import pytest
import torch

import kda_decode_recurrence_gb300 as kda

from _paged import cumulative, verify
from _parity import Guarded

pytestmark = pytest.mark.gpu


def draws(n, V, seed, near=0.7, point=False, peak=2.5):
    g = torch.Generator().manual_seed(seed)
    N, B = sum(n), len(n)
    target = torch.softmax(peak * torch.randn(N + B, V, generator=g), -1)
    cu = cumulative(n)
    rows = [cu[b] + b + i for b in range(B) for i in range(n[b])]
    draft = torch.softmax(target[rows].clamp_min(1e-30).log() + near * torch.randn(N, V, generator=g), -1)
    # 0 or at least 2^-36, so that the reference's integers hold every value exactly
    target, draft = [torch.where(x < 2.0 ** -36, torch.zeros(()), x) for x in (target, draft)]
    tokens = (torch.multinomial(draft, 1, generator=g)[:, 0] if N else torch.zeros(0)).to(torch.int32)
    return dict(target=target, draft=None if point else draft, draft_tokens=tokens,
                accept_u=torch.rand(N, generator=g), sample_u=torch.rand(B, generator=g), n=n)


def call(d, pad=0, status_expected=0):
    n = d["n"]
    N, B, V = sum(n), len(n), d["target"].shape[1]

    def rows(x):
        if x is None:
            return None
        wide = torch.full((x.shape[0], V + pad), float("nan"), device="cuda")
        wide[:, :V] = x.cuda()
        return wide[:, :V]

    tokens = Guarded((N + B,), torch.int32, fill=-7)
    accepted = Guarded((B,), torch.int32, fill=-7)
    status = kda.kda_verify_draft(tokens.t, accepted.t, rows(d["target"]), rows(d["draft"]), d["draft_tokens"].cuda(),
                                  d["accept_u"].cuda(), d["sample_u"].cuda(),
                                  torch.tensor(cumulative(n), dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(status.item()) == status_expected and tokens.intact() and accepted.intact()
    return tokens.t.cpu().numpy(), accepted.t.cpu().numpy()


def check(d, **kw):
    tokens, accepted = call(d, **kw)
    want = verify(*[None if d[k] is None else d[k].numpy() for k in ("target", "draft", "draft_tokens", "accept_u", "sample_u")], d["n"])
    assert np.array_equal(accepted, want[1])
    assert np.array_equal(tokens, want[0])
    return tokens, accepted


@pytest.mark.parametrize("V", [1, 2, 31, 33, 64, 1000, 4099, 32001])
@pytest.mark.parametrize("n", [[0], [1], [4], [0, 1, 7, 0, 3], [40, 2]])
@pytest.mark.parametrize("point", [False, True], ids=["probs", "point"])
def test_against_the_definition(V, n, point):
    check(draws(n, V, seed=V + len(n), point=point))


def test_padded_rows_and_a_large_vocabulary():
    check(draws([3, 0, 7], 131071, seed=3, peak=1.0), pad=5)
    check(draws([2, 2], 200000, seed=4, peak=0.1, near=0.1))


def test_acceptance_is_common_and_rejection_too():
    n = [5] * 60
    _, accepted = check(draws(n, 500, seed=5))
    assert 0 in accepted and 5 in accepted and len(set(accepted.tolist())) >= 4


def test_borders_of_the_comparison():
    """u q = p exactly is no acceptance; the next smaller u accepts."""
    for u, taken in ((0.5, 0), (float(np.nextafter(np.float32(0.5), np.float32(0))), 1)):
        d = dict(target=torch.tensor([[0.25, 0.75], [1.0, 0.0]]), draft=torch.tensor([[0.5, 0.5]]),
                 draft_tokens=torch.tensor([0], dtype=torch.int32), accept_u=torch.tensor([u]),
                 sample_u=torch.tensor([0.0]), n=[1])
        _, accepted = check(d)
        assert accepted[0] == taken
    # fp32 would round u q up to p here
    u, q = np.float32(1 - 2.0 ** -24), np.float32(1 - 2.0 ** -24)
    p = np.float32(1 - 2.0 ** -23)
    d = dict(target=torch.tensor([[float(p), 1 - float(p)], [1.0, 0.0]]), draft=torch.tensor([[float(q), 1 - float(q)]]),
             draft_tokens=torch.tensor([0], dtype=torch.int32), accept_u=torch.tensor([float(u)]),
             sample_u=torch.tensor([0.0]), n=[1])
    check(d)


@pytest.mark.parametrize("V", [64, 1024, 65536])
def test_borders_of_the_draw(V):
    """Equal dyadic weights: C(v) = (v + 1) / V exactly, u on the border between two entries."""
    for k in (0, 1, V // 2, V - 1):
        d = dict(target=torch.full((1, V), 1.0 / V), draft=None, draft_tokens=torch.zeros(0, dtype=torch.int32),
                 accept_u=torch.zeros(0), sample_u=torch.tensor([k / V]), n=[0])
        tokens, _ = check(d)
        assert tokens[0] == k


def test_draws_skip_entries_without_weight():
    p = torch.zeros(1, 3000)
    p[0, [7, 1999, 2998]] = torch.tensor([0.25, 0.5, 0.25])
    for u, want in ((0.0, 7), (0.2499, 7), (0.25, 1999), (0.75, 2998), (1 - 2.0 ** -24, 2998)):
        d = dict(target=p, draft=None, draft_tokens=torch.zeros(0, dtype=torch.int32), accept_u=torch.zeros(0),
                 sample_u=torch.tensor([u]), n=[0])
        tokens, _ = check(d)
        assert tokens[0] == want


def test_what_is_not_a_number_weighs_nothing():
    d = draws([1, 0], 700, seed=8)
    d["accept_u"][0] = 1 - 2.0 ** -24
    d["draft"][0, d["draft_tokens"][0]] = 1.0        # rejected unless the target is as sure
    d["target"][0, ::3] = float("nan")
    check(d)
    d["target"][2] = 0.0                             # nothing to draw from
    tokens, _ = call(d, status_expected=kda.DEV_BAD_PROB)
    assert tokens[2] == -1
    d["target"][2, 5] = float("inf")
    tokens, _ = call(d, status_expected=kda.DEV_BAD_PROB)
    assert tokens[2] == -1


def test_bad_tokens_and_ranges_are_reported():
    d = draws([3, 2], 100, seed=9)
    d["draft_tokens"][1] = 100
    d["draft_tokens"][3] = -1
    d["accept_u"][:] = 0.0
    tokens, accepted = call(d, status_expected=kda.DEV_BAD_TOKEN)
    want = verify(*[d[k].numpy() for k in ("target", "draft", "draft_tokens", "accept_u", "sample_u")], d["n"])
    assert np.array_equal(tokens, want[0]) and np.array_equal(accepted, want[1])
    assert accepted[0] <= 1 and accepted[1] == 0
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in draws([3, 2], 100, seed=9).items()}
    tokens, accepted = [torch.full((s,), -7, dtype=torch.int32, device="cuda") for s in (7, 2)]
    for cu, skipped in (([0, 3, 99], 1), ([0, -1, 5], 0), ([4, 3, 5], 0)):
        tokens.fill_(-7)
        accepted.fill_(-7)
        status = kda.kda_verify_draft(tokens, accepted, d["target"], d["draft"], d["draft_tokens"], d["accept_u"],
                                      d["sample_u"], torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert int(status.item()) == kda.DEV_BAD_SEQLEN
        assert int(accepted[skipped]) == -7


def test_the_drawn_tokens_follow_the_target():
    """10,000 requests over one pair of distributions: the frequency of each first token
    is the target's within 5 standard deviations."""
    B, V = 10000, 12
    g = torch.Generator().manual_seed(10)
    p, q = [torch.softmax(1.5 * torch.randn(V, generator=g), -1) for _ in range(2)]
    drafts = torch.multinomial(q, B, replacement=True, generator=g).to(torch.int32)
    d = dict(target=p.repeat(2 * B, 1), draft=q.repeat(B, 1), draft_tokens=drafts, accept_u=torch.rand(B, generator=g),
             sample_u=torch.rand(B, generator=g), n=[1] * B)
    tokens, _ = call(d)
    seen = np.bincount(tokens[::2], minlength=V) / B
    p = p.numpy().astype(float)
    assert np.all(np.abs(seen - p) <= 5 * np.sqrt(p * (1 - p) / B))


def test_the_sums_hold_on_a_border_of_a_large_vocabulary():
    """Long sums of weights that span many octaves, the target u' times the
    sum at 2^-37 of itself before or behind a border: further than the sums' error lets it
    move (less than 2^-38 of the sum before the border and of the target).  All lanes add the same
    sequence, so that no error averages out."""
    V, length = 1 << 27, 1 << 14
    g = np.random.default_rng(6)
    s = (np.exp(3 * g.standard_normal((2, 64, length))) * 2.0 ** -32).astype(np.float32)
    s = s[0, 44], s[1, 59]                                   # (whose plain pair sums were off by 2^-34)
    s = np.stack([s[0], s[1] * np.float32(0.9 * s[0].sum(dtype=float) / s[1].sum(dtype=float))])
    s[0, -1] = s[1, 0] = np.float32(2.0 ** -32)                # at the border
    rows = [torch.from_numpy(x).cuda().view(-1, 1, 4).expand(-1, 32, 4).reshape(1, -1) for x in s]
    weights = torch.cat([x.expand(V // 2 // x.shape[1], -1).reshape(1, -1) for x in rows], 1)
    unit = 2.0 ** 110                                           # every weight a whole number of 1 / unit
    each = V // 2 // length
    halves = [sum(int(float(y) * unit) for y in x) * each for x in s]
    spare = weights[0, V - 3:].cpu().numpy()                    # three entries that make up the difference
    for sign, drawn in ((1, V // 2), (-1, V // 2 - 1)):
        rest = halves[0] + sign * (halves[0] >> 36) - (halves[1] - sum(int(float(y) * unit) for y in spare))
        fill = []
        for _ in range(3):
            y = np.float32(rest / unit)
            if int(float(y) * unit) > rest:                     # (rounded down: no weight is negative)
                y = np.nextafter(y, np.float32(0))
            fill.append(y)
            rest -= int(float(y) * unit)
        assert abs(rest) <= halves[0] >> 60
        weights[0, V - 3:] = torch.tensor(fill)
        tokens = torch.zeros(1, dtype=torch.int32, device="cuda")
        accepted = torch.zeros(1, dtype=torch.int32, device="cuda")
        none, half = torch.zeros(0, device="cuda"), torch.full((1,), 0.5, device="cuda")
        status = kda.kda_verify_draft(tokens, accepted, weights, None, none.int(), none, half,
                                      torch.zeros(2, dtype=torch.int32, device="cuda"))
        assert int(status) == 0 and int(tokens) == drawn


@pytest.mark.parametrize("at", [0, 3, 31, 32, 50, 69])
@pytest.mark.parametrize("point", [False, True], ids=["probs", "point"])
def test_a_bad_token_is_reported_wherever_it_stands(at, point):
    """Also behind a draft that was rejected, however far."""
    d = draws([70, 2], 50, seed=12, point=point)
    d["accept_u"][0] = 1.0 - 2.0 ** -24          # draft 0 of request 0: proposed with more than the target has
    x = int(d["draft_tokens"][0])
    d["target"][0] = (1.0 - torch.nn.functional.one_hot(torch.tensor(x), 50).float()) / 49
    for bad in (50, -1, -2 ** 31):
        d["draft_tokens"][at] = bad
        tokens, accepted = call(d, status_expected=kda.DEV_BAD_TOKEN)
        want = verify(*[None if d[k] is None else d[k].numpy() for k in ("target", "draft", "draft_tokens", "accept_u", "sample_u")], d["n"])
        assert accepted[0] == 0 and np.array_equal(tokens, want[0]) and np.array_equal(accepted, want[1])


@pytest.mark.parametrize("B", [304, 305, 400, 608, 609, 800, 1216, 1217, 2000])
@pytest.mark.parametrize("V", [257, 1024])
def test_many_requests_of_every_cluster_size(B, V):
    """Clusters of 8, 4, 2 and 1 CTAs per request, compared exactly."""
    check(draws([i % 3 for i in range(B)], V, seed=B, point=V == 257), pad=0 if V == 1024 else 3)
