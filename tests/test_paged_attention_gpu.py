"""kda_paged_attention against softmax attention in 64 bits, position by position
(tolerances: see _paged.attention).  Rows of the cache that no position in use owns
hold NaN throughout."""
import pytest
import torch

import kda_decode_recurrence_gb300 as kda

from _paged import Case, U_BF16, U_F32, attention, cumulative
from _parity import Guarded

pytestmark = pytest.mark.gpu


def queries(case, H, seed=1, amplitude=1.0):
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn(case.T, H + 2, case.D, generator=g) * amplitude).to(torch.bfloat16).cuda()
    return wide[:, :H]                      # tokens strided by (H + 2) D


def attend(case, q, causal=True, window=0, scale=None, max_tokens=None, table=None, with_lse=True,
           seq_lens=None, stream=None):
    """The call on guarded outputs and workspace; returns (out, lse, status)."""
    T, H, D = q.shape
    out = Guarded((T, H, D), torch.bfloat16, fill=float("nan"))
    lse = Guarded((T, H), torch.float32, fill=float("nan"))
    most = max(case.n) if max_tokens is None else max_tokens
    work = Guarded((kda.paged_attention_workspace_size(case.B, T, most, H, case.HKV, D),), torch.uint8, fill=0xFF)
    caches, scales = case.args()
    status = kda.kda_paged_attention(out.t, q, *caches, case.cu, case.seq_lens if seq_lens is None else seq_lens,
                                     case.table if table is None else table, most, scale=scale, causal=causal,
                                     window=window, **scales, lse=lse.t if with_lse else None, workspace=work.t,
                                     stream=stream)
    torch.cuda.synchronize()
    assert out.intact() and lse.intact() and work.intact()
    return out.t, lse.t, int(status.item())


def check(case, q, causal=True, window=0, scale=None, table=None, **kw):
    out, lse, status = attend(case, q, causal, window, scale, table=table, **kw)
    assert status == 0
    want, wlse, tol, ltol = attention(case, q, q.shape[2] ** -0.5 if scale is None else scale, causal, window, table)
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), f"off by {float((off / tol.clamp_min(1e-300)).max()):.3g} tolerances"
    empty = torch.isneginf(wlse)
    assert torch.equal(torch.isneginf(lse), empty) and bool((out[empty] == 0).all())
    off = (lse.double() - wlse)[~empty].abs()
    assert bool((off <= ltol[~empty]).all()), f"lse off by {float((off / ltol[~empty]).max()):.3g} tolerances"


SHAPES = [
    # single tokens: one key, page and tile edges
    dict(n=[1], lens=[1], H=1, HKV=1, D=128, page=16),
    dict(n=[1] * 7, lens=[1, 15, 16, 17, 63, 64, 65], H=8, HKV=2, D=128, page=16),
    dict(n=[1] * 5, lens=[127, 128, 129, 255, 257], H=12, HKV=1, D=128, page=64),
    dict(n=[1] * 4, lens=[300, 1, 700, 33], H=6, HKV=2, D=64, page=32),
    dict(n=[1, 1], lens=[1500, 2], H=32, HKV=2, D=128, page=128),
    dict(n=[1], lens=[5000], H=4, HKV=1, D=64, page=16),
    dict(n=[1], lens=[4099], H=16, HKV=1, D=128, page=64),
    # drafted windows, empty requests, padding (more new tokens than positions)
    dict(n=[1, 2, 3, 4, 5, 6, 7, 8], lens=[9, 2, 100, 64, 130, 6, 65, 257], H=8, HKV=2, D=128, page=16),
    dict(n=[0, 5, 0, 3], lens=[0, 40, 12, 3], H=5, HKV=5, D=64, page=16),
    dict(n=[4, 6, 3], lens=[2, 0, 50], H=4, HKV=2, D=128, page=16),
    dict(n=[8, 8], lens=[520, 41], H=24, HKV=2, D=128, page=32),
    dict(n=[7], lens=[300], H=7, HKV=1, D=64, page=64),
    # chunks: rows of several tiles, with and without a cached prefix
    dict(n=[40], lens=[40], H=4, HKV=2, D=128, page=16),
    dict(n=[100, 33], lens=[230, 33], H=8, HKV=2, D=128, page=64),
    dict(n=[130], lens=[390], H=2, HKV=2, D=64, page=32),
    dict(n=[257], lens=[257], H=3, HKV=1, D=128, page=128),
    dict(n=[70, 1, 0, 20], lens=[64, 900, 5, 300], H=12, HKV=1, D=128, page=16),
    dict(n=[65, 2], lens=[80, 90], H=20, HKV=4, D=64, page=16),
]
IDS = [f"n{max(s['n'])}_L{max(s['lens'])}_H{s['H']}_{s['HKV']}_D{s['D']}_p{s['page']}" for s in SHAPES]


def make(shape, **kw):
    shape = dict(shape)
    H = shape.pop("H")
    case = Case(**shape, **kw)
    return case, queries(case, H)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_causal(shape, cache):
    case, q = make(shape, cache=cache, seed=11)
    check(case, q)


@pytest.mark.parametrize("window", [1, 16, 100, 129])
@pytest.mark.parametrize("shape", [SHAPES[i] for i in (1, 4, 5, 7, 9, 13, 15, 16)], ids=lambda s: f"L{max(s['lens'])}")
def test_window(shape, window):
    case, q = make(shape, cache="bf16" if window % 2 else "e4m3", seed=12)
    check(case, q, window=window)


@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("shape", [SHAPES[i] for i in (0, 4, 8, 9, 13, 16)], ids=lambda s: f"L{max(s['lens'])}")
def test_not_causal(shape, window):
    case, q = make(shape, cache="e4m3" if window else "bf16", seed=13)
    check(case, q, causal=False, window=window)


@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[7], SHAPES[13]], ids=["token", "window", "chunk"])
def test_large_scores_and_another_scale(shape):
    """Scores in the hundreds: one weight near 1, the rest below fp32's range."""
    case, q = make(shape, seed=14)
    check(case, q * 8, scale=0.5)
    check(case, q, scale=-0.1)
    check(case, q, scale=0.0)


@pytest.mark.parametrize("shape", [SHAPES[3], SHAPES[10], SHAPES[14]], ids=["token", "window", "chunk"])
def test_values_of_extreme_size(shape):
    """Values near bf16's ends: the weights' product with V neither overflows nor vanishes."""
    for amplitude in (1e-30, 1e30):
        case, q = make(shape, seed=15)
        v = case.tensors["v"][0]
        v.copy_((v.float() * amplitude).to(torch.bfloat16))
        check(case, q)
    case, q = make(shape, cache="e4m3", seed=15)
    for amplitude in (1e-20, 1e20):
        scale = case.tensors["v"][1].clone()
        case.tensors["v"][1].mul_(amplitude)
        check(case, q)
        case.tensors["v"][1].copy_(scale)


@pytest.mark.parametrize("n,lens,G", [(1, 300, 4), (6, 300, 8), (90, 300, 4), (150, 150, 2)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_not_a_number_in_masked_places(n, lens, G, cache):
    """K and V of positions outside a token's window or after it hold NaN and infinity,
    and pages wholly before the window are gone: tokens that do not see them are as before."""
    window = 64
    case, q = make(dict(n=[n, n], lens=[lens, lens - 3], H=2 * G, HKV=2, D=128, page=16), cache=cache, seed=16)
    want, wlse, _ = attend(case, q, window=window)
    table = case.table.clone()
    for b in range(2):
        first = max(0, case.lens[b] - n - window + 1)          # the first position any token sees
        table[b, :first // 16] = -1
        for pos in range(first // 16 * 16, first):
            for name, bad in (("k", float("nan")), ("v", float("inf"))):
                x, s = case.tensors[name]
                row = (int(case.table[b, pos // 16]), slice(None), pos % 16)
                if s is None:
                    x[row] = bad
                else:
                    s[row] = bad
    out, lse, status = attend(case, q, window=window, table=table)
    assert status == 0
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("n,lens,G", [(5, 70, 4), (8, 200, 8), (90, 300, 4), (150, 150, 2), (300, 300, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_value_reaches_only_the_tokens_that_see_it(n, lens, G, bad):
    """A later token's V that is not finite: earlier tokens of the chunk are as before."""
    case, q = make(dict(n=[n], lens=[lens], H=2 * G, HKV=2, D=128, page=16), seed=17)
    want, wlse, _ = attend(case, q)
    i = (2 * n) // 3                                            # its position becomes bad
    pos = lens - n + i
    case.tensors["v"][0][int(case.table[0, pos // 16]), :, pos % 16, 5] = bad
    out, lse, status = attend(case, q)
    assert status == 0
    assert torch.equal(out[:i], want[:i]) and torch.equal(lse, wlse)
    keep = torch.arange(128, device="cuda") != 5
    assert torch.equal(out[i:][..., keep], want[i:][..., keep])
    assert not bool(torch.isfinite(out[i:][..., 5]).any())


def test_without_lse_and_on_another_stream():
    case, q = make(SHAPES[13], seed=18)
    want, _, _ = attend(case, q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out, _, status = attend(case, q, with_lse=False, stream=stream)
    assert status == 0 and torch.equal(out, want)


def test_max_tokens_only_chooses_kernels():
    """A larger bound than needed: the same values, within the tolerance of either."""
    for shape in (SHAPES[2], SHAPES[7], SHAPES[16]):
        case, q = make(shape, seed=19)
        for most in (max(case.n), max(case.n) + 1, 5000):
            check(case, q, max_tokens=most)


def test_same_call_same_bits_and_graph_replay():
    for shape in (SHAPES[5], SHAPES[7], SHAPES[13], SHAPES[16]):
        case, q = make(shape, seed=20)
        want, wlse, _ = attend(case, q)
        again, alse, _ = attend(case, q)
        assert torch.equal(want, again) and torch.equal(wlse, alse)
        caches, scales = case.args()
        out, lse = torch.zeros_like(want), torch.zeros_like(wlse)
        work = torch.empty(kda.paged_attention_workspace_size(case.B, case.T, max(case.n), q.shape[1], case.HKV, case.D),
                           dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.kda_paged_attention(out, q, *caches, case.cu, case.seq_lens, case.table, max(case.n), **scales,
                                    lse=lse, workspace=work, dev_status=status)
        for _ in range(2):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(lse, wlse) and int(status.item()) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,D", [(1024, 128), (1024, 64), (24, 128), (24, 64)])
def test_same_bits_when_copies_arrive_late(n, D, cache):
    """Long caches read through a cold L2 and through a warm one: the order in which copies
    arrive must not show."""
    lens, HKV, page = 12000, 4, 64
    g = torch.Generator(device="cuda").manual_seed(25)
    pages = 4 * (-(-lens // page))
    k, v = [torch.randn(pages, HKV, page, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    scales = {}
    if cache == "e4m3":
        k, v = [(x.float() * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for x in (k, v)]
        scales = {s: torch.rand(pages, HKV, page, device="cuda", generator=g) * 0.01 + 0.002 for s in ("k_scale", "v_scale")}
    table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(4, -1)
    q = torch.randn(4 * n, 4 * HKV, D, device="cuda", generator=g).to(torch.bfloat16)
    cu = torch.arange(5, dtype=torch.int32, device="cuda") * n
    seq = torch.full((4,), lens, dtype=torch.int32, device="cuda")
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    first = None
    for trial in range(8):
        if trial % 2 == 0:
            flush.fill_(trial)
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        assert int(kda.kda_paged_attention(out, q, k, v, cu, seq, table, n, **scales, lse=lse).item()) == 0
        if first is None:
            first = (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), f"trial {trial}"


@pytest.mark.parametrize("shape", [SHAPES[3], SHAPES[7], SHAPES[13]], ids=["token", "window", "chunk"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_bad_page_counts_as_zero_rows(shape, cache):
    case, q = make(shape, cache=cache, seed=21)
    table = case.table.clone()
    table[0, 0] = case.num_pages
    table[case.B - 1, 0] = -5
    out, lse, status = attend(case, q, table=table)
    assert status == kda.DEV_BAD_PAGE
    want, wlse, tol, ltol = attention(case, q, case.D ** -0.5, table=table)
    assert bool(((out.double() - want).abs() <= tol).all())
    some = ~torch.isneginf(wlse)
    assert bool(((lse.double() - wlse)[some].abs() <= ltol[some]).all())


def test_bad_lengths_are_reported_and_skipped():
    case, q = make(SHAPES[13], seed=22)       # n = 100, 33
    want, _, _ = attend(case, q)
    lens = case.seq_lens.clone()
    lens[1] = case.max_pages * case.page + 1
    out, _, status = attend(case, q, seq_lens=lens)
    assert status == kda.DEV_BAD_SEQLEN
    assert torch.equal(out[:100], want[:100]) and bool(torch.isnan(out[100:]).all())
    out, _, status = attend(case, q, max_tokens=50)
    assert status == kda.DEV_BAD_SEQLEN
    assert bool(torch.isnan(out[:100]).all()) and bool(torch.isfinite(out[100:]).all())


@pytest.mark.parametrize("n", [1, 40])
def test_offsets_beyond_32_bits(n):
    """Pages past 2^31 elements of the cache (the last ones of 4.9 GB)."""
    small, q = make(dict(n=[n], lens=[200], H=8, HKV=8, D=128, page=128), seed=23, junk=0.0)
    pages = 18400
    big = [torch.zeros(pages, 8, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for i, x in enumerate(big):
        x[-small.num_pages:] = small.tensors["kv"[i]][0]
    table = torch.where(small.table >= 0, small.table + pages - small.num_pages, small.table)
    want, _, _ = attend(small, q)
    out = torch.empty_like(want)
    status = kda.kda_paged_attention(out, q, *big, small.cu, small.seq_lens, table, n)
    assert int(status.item()) == 0 and torch.equal(out, want)


def test_many_requests():
    """More requests than threads of a block, lengths from 0."""
    g = torch.Generator().manual_seed(24)
    lens = torch.randint(0, 60, (700,), generator=g).tolist()
    case, q = make(dict(n=[min(1, x) for x in lens], lens=lens, H=2, HKV=1, D=64, page=16), seed=24)
    check(case, q)


# n, lens and query heads of single tokens, windows and chunks (of one and two row tiles)
KERNELS = [(1, 300, 4), (5, 200, 4), (60, 300, 4), (150, 150, 2), (300, 300, 1)]


@pytest.mark.parametrize("n,lens,G", KERNELS)
@pytest.mark.parametrize("amplitude", [2.0 ** -115, 2.0 ** -90, 2.0 ** 120])
def test_value_scales_at_both_ends(n, lens, G, amplitude):
    """Value scales near the ends of fp32's range (here 2^-10 .. 2^-5 times the amplitude): the
    sum of the weights keeps within it.  At 2^-115 the weights' product with a scale has few
    bits left, and only the log-sum is compared."""
    case, q = make(dict(n=[n], lens=[lens], H=2 * G, HKV=2, D=128, page=16), cache="e4m3", seed=31)
    case.tensors["v"][1].mul_(amplitude)
    if amplitude >= 2.0 ** -90:
        check(case, q)
        return
    out, lse, status = attend(case, q)
    _, want, _, tol = attention(case, q, case.D ** -0.5)
    assert status == 0 and bool(((lse.double() - want).abs() <= tol).all())
    assert bool((out.double().abs() <= case.dense("v", 0).abs().max()).all())


@pytest.mark.parametrize("n,lens,G", KERNELS[1:])
def test_a_row_that_is_not_finite_reaches_only_the_tokens_that_see_it(n, lens, G):
    """A later token's V row with a NaN, appended to an e4m3 cache: earlier tokens are as
    before, and the ones that see it are not numbers."""
    case, q = make(dict(n=[n], lens=[lens], H=2 * G, HKV=2, D=128, page=16), cache="e4m3", seed=32)
    i = (2 * n) // 3
    k, v = (torch.randn(n, 2, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(s)).to(torch.bfloat16)
            for s in (1, 2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    (kc, vc), scales = case.args()

    def append():
        kda.kda_cache_append(kc, vc, k, v, case.cu, case.seq_lens, case.table, dev_status=status, **scales)

    append()
    want, wlse, _ = attend(case, q)
    v[i, 1, 7] = float("nan")
    append()
    out, lse, bits = attend(case, q)
    assert bits == 0 and int(status) == 0
    pos = lens - n + i
    assert not bool(vc[int(case.table[0, pos // 16]), 1, pos % 16].view(torch.uint8).any())  # codes of 0
    assert torch.equal(out[:i], want[:i]) and torch.equal(lse[:i], wlse[:i])
    assert torch.equal(out[:, :G], want[:, :G])
    assert bool(torch.isnan(out[i:, G:]).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,most,G", [([197, 3], 100, 4), ([195, 5], 100, 2), ([1, 199, 8, 32], 60, 1)])
def test_a_request_that_is_too_long_leaves_the_others_served(n, most, G, cache):
    """T = B max_tokens, yet not every request has max_tokens tokens: one has more (and is
    skipped), the short ones are as alone."""
    assert sum(n) == len(n) * most
    case, q = make(dict(n=n, lens=[x + 150 for x in n], H=2 * G, HKV=2, D=128, page=16), cache=cache, seed=41)
    out, lse, status = attend(case, q, max_tokens=most)
    assert status == kda.DEV_BAD_SEQLEN
    want, wlse, tol, ltol = attention(case, q, q.shape[2] ** -0.5)
    at = cumulative(n)
    for b, x in enumerate(n):
        rows = slice(at[b], at[b + 1])
        if x > most:
            assert bool(torch.isnan(out[rows]).all()) and bool(torch.isnan(lse[rows]).all())
        else:
            assert bool(((out[rows].double() - want[rows]).abs() <= tol[rows]).all())
            assert bool(((lse[rows].double() - wlse[rows]).abs() <= ltol[rows]).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("full,n,G", [(1, [1, 0, 1], 4), (6, [1, 3, 6], 2), (24, [24, 2, 9], 4), (150, [3, 150, 60], 2)])
def test_offsets_that_do_not_span_the_tokens_are_reported(full, n, G, cache):
    """cu[B] < T (a graph captured with full windows, replayed with shorter ones) and cu[0] > 0
    set the status; the requests are served all the same."""
    B = len(n)
    case, q = make(dict(n=n, lens=[x + 100 for x in n], H=2 * G, HKV=2, D=128, page=16), cache=cache, seed=42)
    want, wlse, tol, ltol = attention(case, q, 128 ** -0.5)
    caches, scales = case.args()
    shape = (B * full, 2 * G, 128)
    wide = torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    out, lse = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(shape[:2], 7.0, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * full
    lens = torch.full((B,), full + 50, dtype=torch.int32, device="cuda").clamp_max(case.max_pages * 16)
    work = torch.empty(kda.paged_attention_workspace_size(B, B * full, full, 2 * G, 2, 128), dtype=torch.uint8, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_paged_attention(out, wide, *caches, cu, lens, case.table, full, **scales, lse=lse, workspace=work,
                                dev_status=word)
    lens.copy_(case.seq_lens)
    for first in (0, 1):                         # cu[0] = 1: a row in front that is nobody's
        if first + sum(n) > B * full:
            continue
        cu.copy_(case.cu + first)
        rows = slice(first, first + sum(n))
        wide[rows] = q
        out.fill_(7.0)
        word.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert int(word) == kda.DEV_BAD_SEQLEN
        assert bool(((out[rows].double() - want).abs() <= tol).all())
        assert bool(((lse[rows].double() - wlse).abs() <= ltol).all())
        assert bool((out[:first] == 7).all()) and bool((out[first + sum(n):] == 7).all())


# requests of up to 32 rows over e4m3: the window kernel's
FEW = [dict(n=[1, 1], lens=[300, 77], H=16, HKV=2, D=128, page=16), dict(n=[4, 4], lens=[200, 70], H=8, HKV=2, D=64, page=32),
       dict(n=[5, 2], lens=[150, 130], H=10, HKV=2, D=128, page=64), dict(n=[60], lens=[150], H=4, HKV=2, D=128, page=16)]
FEW_IDS = ["token", "window16", "window32", "chunk"]


@pytest.mark.parametrize("amplitude", [1.0, 1e-8, 1e-9, 1e-20, 1e12])
@pytest.mark.parametrize("shape", FEW, ids=FEW_IDS)
def test_rows_of_zeros_have_no_say_in_the_weights(shape, amplitude):
    """An appended V row of zeros has the scale 1, a position without a page 0: neither
    takes bits from the weights of values that are much smaller, or larger."""
    for where in ("row", "page"):
        case, q = make(shape, cache="e4m3", seed=46)
        code, scale = case.tensors["v"]
        scale.mul_(amplitude)
        table = case.table.clone()
        if where == "page":
            table[0, 1 if case.lens[0] > case.page else 0] = -7
            out, lse, status = attend(case, q, table=table)
            want, wlse, tol, ltol = attention(case, q, case.D ** -0.5, table=table)
            assert status == kda.DEV_BAD_PAGE
            assert bool(((out.double() - want).abs() <= tol).all()) and bool(((lse.double() - wlse).abs() <= ltol).all())
            continue
        for b in range(case.B):
            for pos in (0, case.lens[b] // 2, case.lens[b] - 1):
                code[int(table[b, pos // case.page]), :, pos % case.page] = 0
                scale[int(table[b, pos // case.page]), :, pos % case.page] = 1.0
        check(case, q)


@pytest.mark.parametrize("factor", [2.0 ** 9, 2.0 ** 40, 2.0 ** -40, 2.0 ** 100])
@pytest.mark.parametrize("shape", FEW, ids=FEW_IDS)
def test_value_rows_of_different_size(shape, factor):
    """Some rows of V far larger or smaller than the others, and 0 in half of their columns:
    those columns come from the other rows alone."""
    case, q = make(shape, cache="e4m3", seed=47)
    code, scale = case.tensors["v"]
    for b in range(case.B):
        for pos in range(0, case.lens[b], 11):
            code.view(torch.uint8)[int(case.table[b, pos // case.page]), :, pos % case.page, ::2] = 0
            scale[int(case.table[b, pos // case.page]), :, pos % case.page] *= factor
    check(case, q)


def whole_rows(case, name, b):
    """Case.dense with all positions at once (every page exists)."""
    x, scale = case.tensors[name]
    pos = torch.arange(case.lens[b], device=x.device)
    page, at = case.table[b, pos // case.page].long(), pos % case.page
    if scale is None:
        return x[page, :, at].double()
    return x.view(torch.uint8)[page, :, at].view(x.dtype).float().double() * scale[page, :, at].double()[..., None]


def whole_attention(case, q, causal, window):
    """_paged.attention with all tokens of a request at once."""
    T, H, D = q.shape
    G, scale = H // case.HKV, D ** -0.5
    parts = [[], [], [], []]
    at = cumulative(case.n)
    for b in range(case.B):
        L, n = case.lens[b], case.n[b]
        k, v = [whole_rows(case, x, b).transpose(0, 1).repeat_interleave(G, 0) for x in "kv"]  # [H, L, D]
        qq = q[at[b]:at[b + 1]].double().transpose(0, 1)                                     # [H, n, D]
        x = scale * qq @ k.transpose(1, 2)
        size = abs(scale) * (qq.abs() @ k.abs().transpose(1, 2))
        j, p = torch.arange(L, device=q.device)[None], (torch.arange(n, device=q.device) + L - n)[:, None]
        see = (j <= p) if causal else (j >= 0).expand(n, L)
        if window:
            see = see & (j > p - window)
        x = x.masked_fill(~see, -float("inf"))
        lse = torch.logsumexp(x, -1)
        P = torch.exp(x - lse[..., None])
        off = (D + 4) * U_F32 * size.masked_fill(~see, 0).amax(-1) + x.masked_fill(~see, 0).abs().amax(-1) * 4 * U_F32 + 2.0 ** -21
        many = see.sum(-1).double()[None]
        out = P @ v
        tol = (U_BF16 + 2 * off + many * U_F32)[..., None] * (P @ v.abs()) + U_BF16 * out.abs()
        ltol = off + many * U_F32 + lse.abs() * 4 * U_F32
        for to, y in zip(parts, (out, lse, tol, ltol)):
            to.append(y.transpose(0, 1))
    return [torch.cat(x) for x in parts]


def whole_check(case, q, causal=True, window=0):
    want, wlse, tol, ltol = whole_attention(case, q, causal, window)
    out, lse, status = attend(case, q, causal, window)
    assert status == 0
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), f"off by {float((off / tol.clamp_min(1e-300)).max()):.3g} tolerances"
    assert bool(((lse.double() - wlse).abs() <= ltol).all())


@pytest.mark.parametrize("H,D", [(8, 128), (16, 64)])
@pytest.mark.parametrize("jump", [2.0 ** 5, 2.0 ** -12, 2.0 ** 60, 2.0 ** -60, 0.0])
def test_value_sizes_that_change_along_the_sequence(H, D, jump):
    """Shares of several key tiles, in which V's scales jump from one tile to a later one."""
    n = [1] * 24 + [2] * 8
    case, q = make(dict(n=n, lens=[2000 + 37 * i for i in range(32)], H=H, HKV=4, D=D, page=64), cache="e4m3", seed=48)
    scale = case.tensors["v"][1]
    for b in range(case.B):
        pages = case.table[b, :-(-case.lens[b] // 64)].long()
        scale[pages[(b % 7) + 3:]] *= jump
        scale[pages[(b % 7) + 9:]] *= 2.0 ** 10
    whole_check(case, q)


@pytest.mark.parametrize("amplitude", [1.0, 2.0 ** -60, 2.0 ** 126])
@pytest.mark.parametrize("n,lens", [(3, 190), (6, 200), (8, 64)])
def test_a_value_scale_that_is_not_finite_reaches_only_the_tokens_that_see_it(n, lens, amplitude):
    """Beside scales of any size, up to the top of fp32's range."""
    case, q = make(dict(n=[n], lens=[lens], H=8, HKV=2, D=128, page=16), cache="e4m3", seed=50)
    case.tensors["v"][1].mul_(amplitude)
    case.tensors["v"][0].view(torch.uint8).bitwise_and_(0x80).bitwise_or_(0x38)     # 1 and -1: no value overflows
    want, wlse, _ = attend(case, q)
    assert bool(torch.isfinite(want).all())
    i, pos = n // 2, lens - n + n // 2
    for bad in (float("inf"), float("nan")):
        case.tensors["v"][1][int(case.table[0, pos // 16]), 1, pos % 16] = bad
        out, lse, status = attend(case, q)
        assert status == 0 and torch.equal(out[:i], want[:i]) and torch.equal(lse, wlse)
        assert torch.equal(out[:, :4], want[:, :4]) and not bool(torch.isfinite(out[i:, 4:]).any())


@pytest.mark.parametrize("factor", [2.0 ** 6, 2.0 ** 12, 2.0 ** 22])
@pytest.mark.parametrize("shape", FEW, ids=FEW_IDS)
def test_scores_of_millions(shape, factor):
    """Scores next to which the logarithm of a value's scale is a fraction of an fp32 step."""
    case, q = make(shape, cache="e4m3", seed=49)
    check(case, q * factor)


@pytest.mark.parametrize("factor", [2.0 ** 22, 2.0 ** 40, 2.0 ** 100, 2.0 ** -100])
@pytest.mark.parametrize("shape", FEW, ids=FEW_IDS)
def test_queries_of_different_size(shape, factor):
    """A head's and a token's queries far larger or smaller than the others: no row of
    queries has a say in another's scores."""
    for which in ("head", "token"):
        case, q = make(shape, cache="e4m3", seed=43)
        q = q.clone()
        if which == "head":
            q[:, 1] = (q[:, 1].float() * factor).to(torch.bfloat16)
        else:
            q[-1:] = (q[-1:].float() * factor).to(torch.bfloat16)
        check(case, q)


@pytest.mark.parametrize("shape", [dict(n=[4, 6], lens=[2, 3], H=4, HKV=2, D=128, page=16),
                                   dict(n=[7, 3], lens=[5, 90], H=8, HKV=2, D=64, page=16),
                                   dict(n=[40], lens=[30], H=4, HKV=2, D=128, page=16)], ids=["16", "32", "chunk"])
def test_queries_of_padding_tokens_have_no_influence(shape):
    """Tokens before position 0 hold anything: huge numbers, infinities, NaN."""
    case, q = make(shape, cache="e4m3", seed=44)
    q = q.contiguous()
    want, wlse, _ = attend(case, q)
    at = cumulative(case.n)
    for junk in (3e38, float("inf"), float("nan")):
        for b in range(case.B):
            q[at[b]:at[b] + max(0, case.n[b] - case.lens[b])] = junk
        out, lse, status = attend(case, q)
        assert status == 0 and torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("big", [2.0 ** 20, 2.0 ** 26, 2.0 ** 45, 2.0 ** 90])
@pytest.mark.parametrize("shape", FEW, ids=FEW_IDS)
def test_entries_of_one_query_of_different_size(shape, big):
    """Where the keys are 0 the queries are huge: the scores come from the small entries alone."""
    case, q = make(shape, cache="e4m3", seed=45)
    q = q.clone()
    q[..., 3] = big
    q[..., 40] = -big
    codes = case.tensors["k"][0].view(torch.uint8)
    codes[..., 3] = 0
    codes[..., 40] = 0x80
    check(case, q)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D", [(24, 128), (32, 64), (43, 128), (64, 128), (65, 64), (100, 128), (128, 128), (128, 64)])
def test_many_query_heads_per_key_head(G, D, cache):
    """Items of five tokens down to one, boxes of up to 128 heads."""
    case, q = make(dict(n=[1, 2, 12], lens=[200, 65, 140], H=G, HKV=1, D=D, page=32), cache=cache, seed=51)
    check(case, q)
    case, q = make(dict(n=[1] * 3, lens=[500, 1, 129], H=2 * G, HKV=2, D=D, page=16), cache=cache, seed=52)
    check(case, q)


LONG = [dict(n=[700], lens=[6000], H=8, HKV=2, D=128, page=64), dict(n=[1500, 33, 400], lens=[1500, 9000, 3100], H=4, HKV=2, D=64, page=16),
        dict(n=[300, 2, 900, 64], lens=[4000, 2500, 900, 64], H=6, HKV=2, D=128, page=128), dict(n=[3001], lens=[3001], H=2, HKV=1, D=128, page=32),
        dict(n=[20] * 40, lens=[1000 + 70 * i for i in range(40)], H=4, HKV=1, D=128, page=64),
        dict(n=[1 + i % 8 for i in range(40)], lens=[900 + 131 * i for i in range(40)], H=8, HKV=2, D=64, page=16)]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1000), (False, 0), (False, 777)])
@pytest.mark.parametrize("shape", LONG, ids=lambda s: f"n{max(s['n'])}_L{max(s['lens'])}")
def test_long_sequences_in_many_pieces(shape, causal, window, cache):
    """Items that several CTAs share, over thousands of positions."""
    case, q = make(shape, cache=cache, seed=53)
    whole_check(case, q, causal, window)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("log2", [28, 31, 33, 36, 60])
@pytest.mark.parametrize("n,lens,G", KERNELS)
def test_scores_of_billions(n, lens, G, log2, cache):
    """Where an fp32 step of a score is hundreds, the largest one's weight is 1 all the same:
    outputs stay within the values."""
    case, q = make(dict(n=[n], lens=[lens], H=2 * G, HKV=2, D=128, page=16), cache=cache, seed=54)
    most = float(max(whole_rows(case, "v", 0).abs().max(), 1))
    out, lse, status = attend(case, q * 2.0 ** log2)
    assert status == 0 and bool((out.double().abs() <= most * (1 + 2 * U_BF16)).all())
    assert bool(torch.isfinite(lse).all())
