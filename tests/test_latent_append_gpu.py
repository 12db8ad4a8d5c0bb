"""kda_latent_append against the formula in 64 bits; rows that no new token names keep their bits."""
import pytest
import torch

import kda_decode_recurrence_gb300 as kda

from _latent import LATENT, ROW, LatentCase
from _paged import U_BF16, U_F32, cumulative
from _parity import Guarded

pytestmark = pytest.mark.gpu


def new_rows(case, seed=3, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(case.T, ROW + 64, generator=g) * torch.exp(spread * torch.randn(case.T, 1, generator=g))
    return x.to(torch.bfloat16).cuda()[:, 64:]     # tokens strided by 640, 128 bytes into the row


def append(case, rows, gamma, eps=1e-5, **kw):
    cache = Guarded(case.cache.shape, torch.bfloat16, like=case.cache)
    if "stream" in kw:  # (the buffers are filled on the current one)
        kw["stream"].wait_stream(torch.cuda.current_stream())
    status = kda.kda_latent_append(cache.t, rows, case.cu, case.seq_lens, kw.pop("table", case.table), gamma=gamma, eps=eps, **kw)
    torch.cuda.synchronize()
    assert cache.intact()
    return cache.t, int(status.item())


def check(case, rows, gamma, got, eps=1e-5, table=None):
    """Every row of the cache: named ones by the formula, the others bit for bit."""
    want = case.cache.clone()
    tol = torch.zeros(want.shape, dtype=torch.float64, device="cuda")
    cu, t = cumulative(case.n), case.table if table is None else table
    exact = want.double()
    for b in range(case.B):
        for i in range(case.n[b]):
            pos = case.lens[b] - case.n[b] + i
            if pos < 0:
                continue
            pg = int(t[b, pos // case.page])
            if not 0 <= pg < case.num_pages:
                continue
            x = rows[cu[b] + i].double()
            y = x.clone()
            if gamma is not None:
                y[:LATENT] = x[:LATENT] * (x[:LATENT].square().mean() + eps) ** -0.5 * gamma.double()
            exact[pg, pos % case.page] = y
            # bf16 of a product of three; the mean of 512 squares (a lane's 16, then five sums) is off by 24
            # roundings, which its root halves; the root, three products, the bf16 itself
            tol[pg, pos % case.page, :LATENT] = (U_BF16 + 17 * U_F32) * y[:LATENT].abs() * (gamma is not None) + (gamma is not None) * 2.0 ** -134
    off = (got.double() - exact).abs()
    same = (got.view(torch.int16) == case.cache.view(torch.int16)) & torch.isnan(exact)
    assert bool(((off <= tol) | same).all())


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("n,lens,page", [
    ([1], [1], 16), ([1] * 7, [1, 15, 16, 17, 63, 64, 65], 16), ([3, 0, 5, 1], [7, 4, 5, 300], 32),
    ([4, 6, 3], [2, 0, 50], 64),                        # padding: tokens before position 0
    ([129, 40], [500, 40], 128), ([9700, 3], [9800, 70], 64)])
def test_rows(n, lens, page, norm):
    case = LatentCase(n, lens, page, seed=len(n))
    rows = new_rows(case)
    gamma = (1 + 0.2 * torch.randn(LATENT)).cuda() if norm else None
    got, status = append(case, rows, gamma)
    assert status == 0
    if sum(n) < 5000:
        check(case, rows, gamma, got)
    else:                                                # in one go: request 0 lies behind position 100
        want = case.cache.double()
        cu = cumulative(n)
        for b in range(2):
            pos = torch.arange(lens[b] - n[b], lens[b], device="cuda")
            x = rows[cu[b]:cu[b + 1]].double()
            if norm:
                x[:, :LATENT] *= (x[:, :LATENT].square().mean(1, keepdim=True) + 1e-5) ** -0.5 * gamma.double()
            want[case.table[b].long()[pos // page], pos % page] = x
        off = (got.double() - want).abs()
        tol = (U_BF16 + 17 * U_F32) * want.abs() if norm else torch.zeros_like(want)
        assert bool(((off <= tol) | torch.isnan(want)).all())


@pytest.mark.parametrize("size,eps", [(2.0 ** 100, 1e-5), (2.0 ** -100, 0.0), (2.0 ** -100, 1e-5), (2.0 ** 60, 0.0), (1.0, 0.0)])
def test_sizes_past_a_square(size, eps):
    """Rows whose squares pass fp32, or fall below it where eps is zero."""
    case = LatentCase([5], [40], 16)
    rows = (torch.randn(5, ROW, generator=torch.Generator().manual_seed(1)) * size).to(torch.bfloat16).cuda()
    gamma = torch.ones(LATENT, device="cuda")
    got, status = append(case, rows, gamma, eps)
    assert status == 0
    check(case, rows, gamma, got, eps)


def test_bad_requests_and_pages():
    case = LatentCase([2, 3, 4], [20, 30, 40], 16)
    rows = new_rows(case)
    table = case.table.clone()
    table[1, 1] = case.num_pages                         # positions 16 .. 31 of request 1
    got, status = append(case, rows, None, table=table)
    assert status == kda.DEV_BAD_PAGE
    check(case, rows, None, got, table=table)
    case.seq_lens[1] = case.max_pages * 16 + 1           # too long: the request is skipped
    got, status = append(case, rows, None)
    assert status == kda.DEV_BAD_SEQLEN
    case.seq_lens[1] = 30
    for b in (0, 2):
        for i in range(case.n[b]):
            pos = case.lens[b] - case.n[b] + i
            assert torch.equal(got[int(case.table[b, pos // 16]), pos % 16], rows[cumulative(case.n)[b] + i])
    assert torch.equal(got[int(case.table[1, 1])].view(torch.int16), case.cache[int(case.table[1, 1])].view(torch.int16))
    cu = case.cu.clone()
    case.cu[3] = 8                                       # offsets that do not span the nine rows
    got, status = append(case, rows, None)
    assert status == kda.DEV_BAD_SEQLEN
    case.cu.copy_(cu)


def test_stream_and_graph():
    case = LatentCase([1] * 40, list(range(1, 41)), 16)
    rows = new_rows(case).contiguous()
    gamma = torch.ones(LATENT, device="cuda")
    want, _ = append(case, rows, gamma)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = append(case, rows, gamma, stream=s)
    used = case.used.cuda()
    assert torch.equal(got[used], want[used])
    cache, status = case.cache.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_latent_append(cache, rows, case.cu, case.seq_lens, case.table, gamma=gamma, dev_status=status)
    rows.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    want, _ = append(case, rows, gamma)
    assert torch.equal(cache[used], want[used]) and int(status.item()) == 0


@pytest.mark.parametrize("size", [2.0 ** -126, 2.0 ** -128, 2.0 ** -131, 2.0 ** -133, 2.0 ** 126])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -91, 2.0 ** -90])
def test_rows_at_the_ends_of_bf16(size, eps):
    """The smallest bf16 numbers, whose reciprocal root mean square passes fp32, and the largest."""
    case = LatentCase([5], [40], 16)
    rows = (torch.randn(5, ROW, generator=torch.Generator().manual_seed(2)).clamp(-3.5, 3.5) * size).to(torch.bfloat16).cuda()
    assert bool((rows[:, :LATENT] != 0).any(1).all())
    gamma = (1 + 0.2 * torch.randn(LATENT, generator=torch.Generator().manual_seed(3))).cuda()
    got, status = append(case, rows, gamma, eps)
    assert status == 0
    check(case, rows, gamma, got, eps)
