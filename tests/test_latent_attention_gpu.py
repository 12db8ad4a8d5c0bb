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
    if "stream" in kw:  # (the buffers are filled on the current one)
        kw["stream"].wait_stream(torch.cuda.current_stream())
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


@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[7], SHAPES[12]], ids=["token", "window", "rows"])
@pytest.mark.parametrize("amplitude,scale", [(1.0, 3.0), (30.0, 1.0), (1e4, 1.0), (1.0, -0.3), (1.0, 0.0)])
def test_scores_of_other_sizes(shape, amplitude, scale):
    case, q = make(shape, seed=31)
    q.mul_(amplitude)
    check(case, q, scale=scale)


@pytest.mark.parametrize("amplitude", [2.0 ** -100, 2.0 ** 50])
def test_latents_of_extreme_size(amplitude):
    case, q = make(SHAPES[7], seed=32)
    case.cache.mul_(amplitude)
    check(case, (q.float() / amplitude).to(torch.bfloat16))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n,lens,H", [(5, 70, 40), (8, 200, 16), (40, 130, 24)])
def test_a_bad_row_reaches_only_the_tokens_that_see_it(n, lens, H, bad):
    """A later token's latent row, or its position part, that is not finite."""
    for at in (5, 300, 540):
        case, q = make(dict(n=[n], lens=[lens], H=H, page=16), seed=33)
        want, wlse, _ = attend(case, q)
        i = (2 * n) // 3
        pos = lens - n + i
        case.cache[int(case.table[0, pos // 16]), pos % 16, at] = bad
        out, lse, status = attend(case, q)
        assert status == 0 and torch.equal(out[:i], want[:i]) and torch.equal(lse[:i], wlse[:i])
        if bad != bad:
            assert bool(torch.isnan(out[i:]).all())


def test_a_bad_node_reaches_only_the_nodes_that_see_it():
    n, L, H = 37, 150, 12
    case, q = make(dict(n=[n], lens=[L], H=H, page=16), seed=34)
    tree = trees([n], seed=3)
    mask = mask_of(tree, 2)
    want, wlse, _ = attend(case, q, mask=mask)
    bad = 11
    pos = L - n + bad
    case.cache[int(case.table[0, pos // 16]), pos % 16] = float("nan")
    out, lse, status = attend(case, q, mask=mask)
    sees = torch.tensor([bad in s for s in tree[0]], device="cuda")
    assert status == 0 and bool(sees.any()) and bool((~sees).any())
    assert torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], wlse[~sees])
    assert bool(torch.isnan(out[sees]).all())


def test_masks_of_nothing_and_of_everything():
    """A mask without bits sees what was cached before; nothing at all without any; one with all bits (those
    past the request's last token are nobody's) is as without causality."""
    case, q = make(dict(n=[5, 33, 1], lens=[5, 133, 40], H=24, page=16), seed=35)
    none = torch.zeros(case.T, 2, dtype=torch.int32, device="cuda")
    out, lse, status = attend(case, q, mask=none)
    assert status == 0
    close(out, lse, reference(case, q, tree=[[set()] * k for k in case.n]))
    assert bool((out[:5] == 0).all()) and bool(torch.isneginf(lse[:5]).all())
    full, flse, _ = attend(case, q, mask=none - 1)
    want, wlse, _ = attend(case, q, causal=False)
    assert torch.equal(full, want) and torch.equal(flse, wlse)
    check(case, q, tree=trees(case.n, seed=9), words=7)


def test_too_many_nodes_for_the_mask_are_reported():
    case, q = make(dict(n=[3, 40, 2], lens=[30, 60, 90], H=8, page=16), seed=36)
    mask = mask_of(trees(case.n), 2)[:, :1].contiguous()
    out, lse, status = attend(case, q, mask=mask)
    assert status == kda.DEV_BAD_SEQLEN
    assert bool(torch.isnan(out[3:43]).all()) and bool(torch.isfinite(out[:3]).all()) and bool(torch.isfinite(out[43:]).all())


def test_without_lse_and_on_another_stream():
    case, q = make(SHAPES[12], seed=37)
    want, _, _ = attend(case, q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out, _, status = attend(case, q, with_lse=False, stream=stream)
    assert status == 0 and torch.equal(out, want)


def test_same_bits_and_graphs_that_share_a_workspace():
    """The same call gives the same bits; two graphs with one workspace, replayed in turn, with other lengths
    than captured."""
    calls = []
    work = torch.empty(kda.latent_attention_workspace_size(8, 100, 64), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for shape, tree in ((SHAPES[7], False), (SHAPES[10], True)):
        case, q = make(shape, seed=38)
        mask = mask_of(trees(case.n), 1) if tree else None
        want, wlse, _ = attend(case, q, mask=mask)
        again, alse, _ = attend(case, q, mask=mask)
        assert torch.equal(want, again) and torch.equal(wlse, alse)
        shorter = torch.clamp(case.seq_lens - 1, min=1)
        less, llse, _ = attend(case, q, mask=mask, seq_lens=shorter)
        lens, out, lse = case.seq_lens.clone(), torch.zeros_like(want), torch.zeros_like(wlse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.kda_latent_attention(out, q, case.cache, case.cu, lens, case.table, tree_mask=mask, lse=lse,
                                     workspace=work, dev_status=status)
        calls.append((graph, lens, case.seq_lens, shorter, out, lse, (want, wlse), (less, llse), case, q, mask))
    for _ in range(3):
        for graph, lens, long, short, out, lse, full, less, *_ in calls:
            for now, (o, e) in ((long, full), (short, less)):
                lens.copy_(now)
                out.zero_()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, o) and torch.equal(lse, e) and int(status.item()) == 0


@pytest.mark.parametrize("n,H", [(1, 128), (1, 16), (6, 32)])
def test_same_bits_when_copies_arrive_late(n, H):
    """Long caches read through a cold L2 and through a warm one."""
    lens, page = 9000, 64
    g = torch.Generator(device="cuda").manual_seed(39)
    pages = 20 * (-(-lens // page))
    cache = torch.randn(pages, page, ROW, device="cuda", generator=g, dtype=torch.bfloat16)
    table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(20, -1)
    q = torch.randn(20 * n, H, ROW, device="cuda", generator=g, dtype=torch.bfloat16)
    cu = torch.arange(21, dtype=torch.int32, device="cuda") * n
    seq = torch.full((20,), lens, dtype=torch.int32, device="cuda")
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    first = None
    for trial in range(8):
        if trial % 2 == 0:
            flush.fill_(trial)
        out, lse = torch.zeros(20 * n, H, LATENT, device="cuda", dtype=torch.bfloat16), torch.zeros(20 * n, H, device="cuda")
        assert int(kda.kda_latent_attention(out, q, cache, cu, seq, table, lse=lse).item()) == 0
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), f"trial {trial}"


@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[7], SHAPES[12]], ids=["token", "window", "rows"])
def test_a_bad_page_counts_as_zero_rows(shape):
    case, q = make(shape, seed=40)
    table = case.table.clone()
    table[0, 0] = case.num_pages
    table[case.B - 1, 0] = -5
    out, lse, status = attend(case, q, table=table)
    assert status == kda.DEV_BAD_PAGE
    close(out, lse, reference(case, q, table=table))


def test_bad_lengths_and_offsets_are_reported_and_skipped():
    """(The others are served, not always with the same bits: the call is cut elsewhere.)"""
    case, q = make(dict(n=[9, 4, 2], lens=[90, 40, 300], H=20, page=16), seed=41)
    want = reference(case, q)

    def served(out, lse, *rows):
        for r in rows:
            close(out[r], lse[r], [x[r] for x in want])

    for bad in (case.max_pages * 16 + 1, -1):
        lens = case.seq_lens.clone()
        lens[1] = bad
        out, lse, status = attend(case, q, seq_lens=lens)
        assert status == kda.DEV_BAD_SEQLEN and bool(torch.isnan(out[9:13]).all())
        served(out, lse, slice(0, 9), slice(13, 15))
    # request 1 ends before it begins (request 2 has row 8 for its first then, which is not looked at)
    out, lse, status = attend(case, q, cu=torch.tensor([0, 9, 8, 15], dtype=torch.int32, device="cuda"))
    assert status == kda.DEV_BAD_SEQLEN
    served(out, lse, slice(0, 8))
    # the last two rows are nobody's
    out, lse, status = attend(case, q, cu=torch.tensor([0, 9, 13, 13], dtype=torch.int32, device="cuda"))
    assert status == kda.DEV_BAD_SEQLEN and bool(torch.isnan(out[13:]).all())
    served(out, lse, slice(0, 13))


@pytest.mark.parametrize("n", [1, 12])
def test_offsets_beyond_32_bits(n):
    """Pages past 2^32 bytes and 2^31 elements of the cache (the last of 5 GB)."""
    small, q = make(dict(n=[n], lens=[400], H=32, page=128), seed=42, junk=0.0)
    pages = 34000
    big = torch.zeros(pages, 128, ROW, dtype=torch.bfloat16, device="cuda")
    big[-small.num_pages:] = small.cache
    table = torch.where(small.table >= 0, small.table + pages - small.num_pages, small.table)
    want, _, _ = attend(small, q)
    out, _, status = attend(small, q, cache=big, table=table)
    assert status == 0 and torch.equal(out, want)
    rows = torch.randn(n, ROW, device="cuda").to(torch.bfloat16)
    kda.kda_latent_append(big, rows, small.cu, small.seq_lens, table, check_device=True)
    at = torch.arange(400 - n, 400, device="cuda")
    assert torch.equal(big[table[0].long()[at // 128], at % 128], rows)


@pytest.mark.parametrize("B", [390, 1300])
def test_many_requests(B):
    """More requests than threads of a block, lengths from 0."""
    g = torch.Generator().manual_seed(43)
    lens = torch.randint(0, 60, (B,), generator=g).tolist()
    case, q = make(dict(n=[min(1, x) for x in lens], lens=lens, H=3, page=16), seed=43)
    check(case, q)


@pytest.mark.parametrize("tree", [False, True])
def test_long_sequences_in_many_pieces(tree):
    """One request over all pairs of CTAs, and one beside it that is a few key tiles."""
    case, q = make(dict(n=[7, 3], lens=[30000, 200], H=40, page=128), seed=44)
    check(case, q, tree=trees(case.n) if tree else None)


def test_empty_calls():
    """No requests, no tokens: nothing is launched."""
    case, q = make(dict(n=[2], lens=[20], H=4, page=16), seed=45)
    out = torch.full((0, 4, LATENT), 1.0, device="cuda", dtype=torch.bfloat16)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert int(kda.kda_latent_attention(out, q[:0], case.cache, zero, case.seq_lens, case.table).item()) == 0
    out, _, status = attend(case, q, cu=zero[:1], seq_lens=zero[:0], table=case.table[:0])
    assert status == 0 and bool(torch.isnan(out).all())


@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("n,lens,pos,H,kind", [
    (1, 70, 20, 16, "causal"), (1, 300, 20, 16, "causal"), (1, 300, 290, 3, "causal"), (5, 200, 100, 16, "causal"),
    (5, 200, 150, 40, "full"), (40, 130, 60, 24, "causal"), (40, 130, 100, 24, "causal"), (3, 9000, 100, 8, "causal"),
    (3, 9000, 8980, 8, "causal"), (2, 9000, 8998, 64, "full"), (37, 150, 20, 12, "tree"), (37, 150, 124, 12, "tree")])
def test_an_infinity_of_weight_zero(n, lens, pos, H, kind, bad):
    """A latent with an infinite entry whose score is -infinity: the products with that entry are 0 x infinity, no number, for
    every token that sees the row, wherever a key tile's border lies; the other entries are as without the row."""
    for col in (7, 400):
        case, q = make(dict(n=[n], lens=[lens], H=H, page=32), seed=46)
        q[..., col] = -(q[..., col].abs() + 0.5) if bad > 0 else q[..., col].abs() + 0.5
        tree = trees(case.n, seed=3) if kind == "tree" else None
        see = seen_by(n, lens, kind == "causal", tree[0] if tree else None)
        case.cache[int(case.table[0, pos // 32]), pos % 32, col] = bad
        out, lse, status = attend(case, q, kind == "causal", mask_of(tree, 2) if tree else None)
        rows, sees = case.dense(0), see[:, pos].clone()
        see[:, pos] = False
        want = softmax64(q, rows[:, None], rows[:, None, :LATENT], see, SCALE)
        assert status == 0 and bool(sees.any()) and bool(torch.isnan(out[sees][..., col]).all())
        out[sees, :, col] = want[0][sees, :, col].to(torch.bfloat16)
        close(out, lse, want)


def test_a_part_of_more_than_a_second():
    """A share that begins with a part of some 1.2 million key tiles (1.4 s at the products' rate) and goes on with seven short
    ones: no warp may give up on a note while it waits for the first.  The pages repeat, and in each period of
    them one row has a score 40 above the others: out is that row, and e^-40 of the others vanishes."""
    page, period, longest = 128, 64, 1 << 30
    lens = [150_000_000] + [400 + 130 * i for i in range(6)] + [longest] * 12
    B, share = len(lens), sum(lens) / 128 / 76                 # key tiles of a pair of CTAs
    assert lens[0] / 128 < share - 200 and lens[0] / 128 > 1.1e6 and share < 1.5e6
    g = torch.Generator(device="cuda").manual_seed(47)
    top = torch.where(torch.rand(ROW, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    cache = torch.randn(period, page, ROW, device="cuda", generator=g).mul_(0.01).to(torch.bfloat16)
    cache[2, 17] = top.to(torch.bfloat16)                      # position 273 of every 8192
    table = (torch.arange(longest // page, dtype=torch.int32, device="cuda") % period).expand(B, -1).contiguous()
    q = (top * 2.0 ** -4).to(torch.bfloat16).expand(B, 1, ROW).contiguous()    # q . top = 36, of the others 0.014 and less
    cu, seq = torch.arange(B + 1, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = torch.full((B, 1, LATENT), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, device="cuda")
    status = kda.kda_latent_attention(out, q, cache, cu, seq, table, scale=40 / 36, lse=lse)
    assert int(status.item()) == 0
    assert torch.equal(out[:, 0], top[:LATENT].to(torch.bfloat16).expand(B, -1))
    count = torch.tensor([-(-(x - 273) // 8192) for x in lens], dtype=torch.float64)
    off = (lse[:, 0].double().cpu() - (40 + torch.log(count))).abs()
    # the score, its factor and the sum's logarithm: a few fp32 roundings of 60; the others: at most 2^30 e^-39
    assert bool((off < 60 * 8 * 2.0 ** -24 + 2.0 ** 30 * 1.2e-17).all())


@pytest.mark.parametrize("n,lens,H", [([4, 6, 3], [2, 0, 50], 40), ([40, 9], [33, 300], 24), ([3, 1, 70], [1, 900, 60], 8)])
@pytest.mark.parametrize("kind", ["causal", "full", "tree"])
def test_queries_of_padding_tokens_have_no_influence(n, lens, H, kind):
    """Tokens before position 0 hold anything: huge numbers, infinities, NaN.  Their rows stand in the same tiles, and in
    the same warps, as those of tokens that see something."""
    case, q = make(dict(n=n, lens=lens, H=H, page=16), seed=48)
    mask = mask_of(trees(n, seed=2), 3) if kind == "tree" else None
    want, wlse, _ = attend(case, q, kind == "causal", mask)
    at = cumulative(n)
    for junk in (3e38, float("inf"), float("nan")):
        for b in range(case.B):
            q[at[b]:at[b] + max(0, n[b] - lens[b])] = junk
        out, lse, status = attend(case, q, kind == "causal", mask)
        assert status == 0 and torch.equal(out, want) and torch.equal(lse, wlse)


def test_infinities_of_many_small_requests():
    """Each reaches the tokens of its own request that see it, whatever shares the kernel's memory with it."""
    g = torch.Generator().manual_seed(49)
    n = torch.randint(1, 7, (420,), generator=g).tolist()
    lens = [k + int(x) for k, x in zip(n, torch.randint(0, 260, (420,), generator=g))]
    case, q = make(dict(n=n, lens=lens, H=10, page=32), seed=49)
    q[..., 300] = -(q[..., 300].abs() + 0.5)
    want, wlse, _ = attend(case, q)
    parts, hit, cu = [], torch.zeros(case.T, dtype=torch.bool, device="cuda"), cumulative(n)
    for b in range(1, case.B, 3):
        pos = lens[b] - n[b] + b % n[b]
        case.cache[int(case.table[b, pos // 32]), pos % 32, 300] = float("inf")
        see, rows = seen_by(n[b], lens[b]), case.dense(b)
        hit[cu[b]:cu[b + 1]] = see[:, pos]
        see[:, pos] = False
        parts.append((softmax64(q[cu[b]:cu[b + 1]], rows[:, None], rows[:, None, :LATENT], see, SCALE), slice(cu[b], cu[b + 1])))
    out, lse, status = attend(case, q)
    assert status == 0 and torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wlse[~hit])
    assert bool(torch.isnan(out[hit][..., 300]).all())
    for exact, at in parts:
        x = out[at].clone()
        x[hit[at], :, 300] = exact[0][hit[at], :, 300].to(torch.bfloat16)
        close(x, lse[at], exact)
