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
    if "stream" in kw:  # (the buffers are filled on the current one)
        kw["stream"].wait_stream(torch.cuda.current_stream())
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


def make(shape, **kw):
    shape = dict(shape)
    H = shape.pop("H")
    case = Case(**shape, **kw)
    return case, queries(case, H)


TREE = dict(n=[37, 9], lens=[150, 300], H=12, HKV=2, D=128, page=16)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_chain_is_as_causal(cache):
    """A chain's mask sees what a causal chunk sees."""
    case, q = make(dict(n=[20, 31], lens=[70, 400], H=16, HKV=2, D=128, page=32), cache=cache, seed=51)
    chain = [[set(range(i + 1)) for i in range(k)] for k in case.n]
    out, lse = check(case, q, chain)
    caches, scales = case.args()
    kda.kda_paged_attention(out, q, *caches, case.cu, case.seq_lens, case.table, 31, **scales, lse=lse, check_device=True)
    # (not the same bits: causal items have fewer key tiles, and so the calls are cut elsewhere)
    close(out, lse, reference(case, q, chain, 128 ** -0.5))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_masks_of_nothing_and_of_everything(cache):
    case, q = make(dict(n=[5, 33, 1], lens=[5, 133, 40], H=8, HKV=2, D=64, page=16), cache=cache, seed=52)
    none = torch.zeros(case.T, 2, dtype=torch.int32, device="cuda")
    out, lse, status = attend(case, q, none)
    assert status == 0
    close(out, lse, reference(case, q, [[set()] * k for k in case.n], 64 ** -0.5))
    assert bool((out[:5] == 0).all()) and bool(torch.isneginf(lse[:5]).all())
    out, lse, status = attend(case, q, none - 1)
    assert status == 0
    close(out, lse, reference(case, q, [[set(range(k))] * k for k in case.n], 64 ** -0.5))
    check(case, q, trees(case.n, seed=9), words=7)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("G", [2, 6])
def test_a_bad_value_reaches_only_the_nodes_that_see_it(bad, G):
    case, q = make(dict(TREE, H=2 * G), seed=53)
    tree = trees(case.n, seed=4)
    mask = mask_of(tree, 2)
    want, wlse, _ = attend(case, q, mask)
    node, L, n = 11, case.lens[0], case.n[0]
    pos = L - n + node
    case.tensors["v"][0][int(case.table[0, pos // 16]), :, pos % 16, 5] = bad
    out, lse, status = attend(case, q, mask)
    sees = torch.tensor([node in s for s in tree[0]] + [False] * case.n[1], device="cuda")
    assert status == 0 and bool(sees.any()) and torch.equal(lse, wlse)
    assert torch.equal(out[~sees], want[~sees])
    keep = torch.arange(128, device="cuda") != 5
    assert torch.equal(out[sees][..., keep], want[sees][..., keep])
    assert not bool(torch.isfinite(out[sees][..., 5]).any())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_bad_key_reaches_only_the_nodes_that_see_it(cache):
    case, q = make(TREE, cache=cache, seed=54)
    tree = trees(case.n, seed=4)
    mask = mask_of(tree, 2)
    want, wlse, _ = attend(case, q, mask)
    node, L, n = 11, case.lens[0], case.n[0]
    pos = L - n + node
    x, s = case.tensors["k"]
    row = (int(case.table[0, pos // 16]), slice(None), pos % 16)
    if s is None:
        x[row] = float("nan")
    else:
        s[row] = float("nan")
    out, lse, status = attend(case, q, mask)
    sees = torch.tensor([node in t for t in tree[0]] + [False] * case.n[1], device="cuda")
    assert status == 0 and torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], wlse[~sees])
    assert bool(torch.isnan(out[sees]).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_scores_of_other_sizes(cache):
    for amplitude, scale in ((30.0, 1.0), (1e4, 1.0), (1.0, -0.3), (1.0, 0.0)):
        case, q = make(TREE, cache=cache, seed=55)
        check(case, (q.float() * amplitude).to(torch.bfloat16), trees(case.n), scale=scale)


def test_on_another_stream_in_a_graph_and_again():
    for cache in ("bf16", "e4m3"):
        case, q = make(TREE, cache=cache, seed=56)
        mask = mask_of(trees(case.n), 2)
        want, wlse, _ = attend(case, q, mask)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        out, _, status = attend(case, q, mask, with_lse=False, stream=stream)
        assert status == 0 and torch.equal(out, want)
        shorter = case.seq_lens - 13
        less, llse, _ = attend(case, q, mask, seq_lens=shorter)
        caches, scales = case.args()
        lens, out, lse = case.seq_lens.clone(), torch.zeros_like(want), torch.zeros_like(wlse)
        work = torch.empty(kda.tree_attention_workspace_size(case.B, case.T, 37, 12, 2, 128), dtype=torch.uint8, device="cuda")
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.kda_tree_attention(out, q, *caches, case.cu, lens, case.table, mask, 37, **scales, lse=lse, workspace=work,
                                   dev_status=word)
        for now, (o, e) in ((case.seq_lens, (want, wlse)), (shorter, (less, llse)), (case.seq_lens, (want, wlse))):
            lens.copy_(now)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, o) and torch.equal(lse, e) and int(word.item()) == 0


def test_bad_pages_lengths_and_offsets():
    case, q = make(dict(n=[9, 4, 2], lens=[90, 40, 300], H=20, HKV=2, D=128, page=16), seed=57)
    tree = trees(case.n)
    mask = mask_of(tree, 1)
    table = case.table.clone()
    table[0, 0], table[2, 3] = case.num_pages, -5
    out, lse, status = attend(case, q, mask, table=table)
    assert status == kda.DEV_BAD_PAGE
    close(out, lse, reference(case, q, tree, 128 ** -0.5, table))
    # (the others are served, not always with the same bits: the call is cut elsewhere)
    exact = reference(case, q, tree, 128 ** -0.5)

    def served(out, lse, *rows):
        for r in rows:
            close(out[r], lse[r], [x[r] for x in exact])

    lens = case.seq_lens.clone()
    lens[1] = case.max_pages * 16 + 1
    out, lse, status = attend(case, q, mask, seq_lens=lens)
    assert status == kda.DEV_BAD_SEQLEN and bool(torch.isnan(out[9:13]).all())
    served(out, lse, slice(0, 9), slice(13, 15))
    out, lse, status = attend(case, q, mask, max_tokens=5)
    assert status == kda.DEV_BAD_SEQLEN and bool(torch.isnan(out[:9]).all())
    served(out, lse, slice(9, 15))
    out, lse, status = attend(case, q, mask, cu=torch.tensor([0, 9, 13, 13], dtype=torch.int32, device="cuda"))
    assert status == kda.DEV_BAD_SEQLEN and bool(torch.isnan(out[13:]).all())
    served(out, lse, slice(0, 13))


def test_offsets_beyond_32_bits():
    """Pages past 2^31 elements of the cache."""
    small, q = make(dict(n=[20], lens=[200], H=16, HKV=8, D=128, page=128), seed=58, junk=0.0)
    pages = 18400
    big = [torch.zeros(pages, 8, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for i, x in enumerate(big):
        x[-small.num_pages:] = small.tensors["kv"[i]][0]
    table = torch.where(small.table >= 0, small.table + pages - small.num_pages, small.table)
    mask = mask_of(trees(small.n), 1)
    want, _, _ = attend(small, q, mask)
    out = torch.empty_like(want)
    status = kda.kda_tree_attention(out, q, *big, small.cu, small.seq_lens, table, mask, 20)
    assert int(status.item()) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_long_sequences_in_many_pieces(cache):
    case, q = make(dict(n=[11, 3], lens=[20000, 200], H=16, HKV=2, D=128, page=128), cache=cache, seed=59)
    check(case, q, trees(case.n))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_a_bad_scale_of_a_value_reaches_only_the_nodes_that_see_it(bad, D):
    case, q = make(dict(TREE, D=D), cache="e4m3", seed=60)
    tree = trees(case.n, seed=4)
    mask = mask_of(tree, 2)
    want, wlse, _ = attend(case, q, mask)
    node, L, n = 11, case.lens[0], case.n[0]
    pos = L - n + node
    case.tensors["v"][1][int(case.table[0, pos // 16]), :, pos % 16] = bad
    out, lse, status = attend(case, q, mask)
    sees = torch.tensor([node in s for s in tree[0]] + [False] * case.n[1], device="cuda")
    assert status == 0 and bool(sees.any()) and torch.equal(lse, wlse)
    assert torch.equal(out[~sees], want[~sees])
    assert not bool(torch.isfinite(out[sees]).any())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_many_small_trees(cache):
    """Several items to each stream of work, most of one key tile."""
    g = torch.Generator().manual_seed(61)
    n = torch.randint(0, 7, (420,), generator=g).tolist()
    lens = [k + int(x) for k, x in zip(n, torch.randint(0, 260, (420,), generator=g))]
    case, q = make(dict(n=n, lens=lens, H=10, HKV=2, D=128, page=32), cache=cache, seed=61)
    check(case, q, trees(n, seed=3))


def test_bad_values_of_many_small_trees():
    """Each reaches the nodes of its own tree that see it, whatever shares the kernel's memory with it."""
    g = torch.Generator().manual_seed(62)
    n = torch.randint(1, 7, (420,), generator=g).tolist()
    lens = [k + int(x) for k, x in zip(n, torch.randint(0, 260, (420,), generator=g))]
    case, q = make(dict(n=n, lens=lens, H=10, HKV=2, D=128, page=32), seed=62)
    tree = trees(n, seed=3)
    mask = mask_of(tree, 1)
    want, wlse, _ = attend(case, q, mask)
    sees = []
    for b in range(case.B):
        if b % 3 == 1:
            node = b % n[b]
            pos = lens[b] - n[b] + node
            case.tensors["v"][0][int(case.table[b, pos // 32]), :, pos % 32, 77] = float("nan")
            sees += [node in s for s in tree[b]]
        else:
            sees += [False] * n[b]
    out, lse, status = attend(case, q, mask)
    sees = torch.tensor(sees, device="cuda")
    assert status == 0 and torch.equal(lse, wlse) and torch.equal(out[~sees], want[~sees])
    keep = torch.arange(128, device="cuda") != 77
    assert torch.equal(out[sees][..., keep], want[sees][..., keep])
    assert bool(torch.isnan(out[sees][..., 77]).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_same_bits_when_copies_arrive_late(cache):
    """Long caches read through a cold L2 and through a warm one, alone and beside calls on other streams."""
    case, q = make(dict(n=[40] * 10, lens=[9001] * 10, H=24, HKV=4, D=128, page=64), cache=cache, seed=63)
    mask = mask_of(trees(case.n), 2)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    first = None
    for trial in range(4):
        if trial % 2 == 0:
            flush.fill_(trial)
        out, lse, status = attend(case, q, mask)
        first = first or (out, lse)
        assert status == 0 and torch.equal(out, first[0]) and torch.equal(lse, first[1]), f"trial {trial}"
    caches, scales = case.args()
    got = [(torch.zeros_like(first[0]), torch.zeros_like(first[1]), torch.cuda.Stream()) for _ in range(3)]
    torch.cuda.synchronize()
    words = [kda.kda_tree_attention(out, q, *caches, case.cu, case.seq_lens, case.table, mask, 40, **scales, lse=lse, stream=s)
             for _ in range(3) for out, lse, s in got]
    torch.cuda.synchronize()
    assert all(int(w.item()) == 0 for w in words)
    assert all(torch.equal(out, first[0]) and torch.equal(lse, first[1]) for out, lse, _ in got)
    close(first[0], first[1], reference(case, q, trees(case.n), 128 ** -0.5))


def test_more_requests_than_threads():
    g = torch.Generator().manual_seed(64)
    n = torch.randint(0, 3, (1300,), generator=g).tolist()
    lens = [k + int(x) for k, x in zip(n, torch.randint(0, 50, (1300,), generator=g))]
    case, q = make(dict(n=n, lens=lens, H=3, HKV=1, D=128, page=16), seed=64)
    check(case, q, trees(n, seed=3))


def test_graphs_that_share_a_workspace():
    """Two captured calls of other sizes, replayed in turns."""
    cases = [make(dict(n=[20, 31], lens=[700, 4000], H=16, HKV=2, D=128, page=32), cache="e4m3", seed=65),
             make(dict(n=[64], lens=[9000], H=32, HKV=8, D=128, page=64), seed=66)]
    need = max(kda.tree_attention_workspace_size(c.B, c.T, max(c.n), q.shape[1], c.HKV, 128) for c, q in cases)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for case, q in cases:
        mask = mask_of(trees(case.n), 2)
        want, wlse, _ = attend(case, q, mask)
        caches, scales = case.args()
        out, lse, word = torch.zeros_like(want), torch.zeros_like(wlse), torch.zeros(1, dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.kda_tree_attention(out, q, *caches, case.cu, case.seq_lens, case.table, mask, max(case.n), **scales,
                                   lse=lse, workspace=work, dev_status=word)
        graphs.append((graph, out, lse, word, want, wlse, mask))  # (the graph reads the mask)
    for turn in range(6):
        for graph, out, lse, *_ in graphs:
            out.zero_()
            lse.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for graph, out, lse, word, want, wlse, _ in graphs:
            assert torch.equal(out, want) and torch.equal(lse, wlse) and int(word.item()) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_bits_do_not_depend_on_what_ran_before(D, cache):
    """126 of a row tile's 128 rows are used (6 heads a group): what the others hold is left over from the call before,
    here of queries of another size.  Trees, and a chunk of the same tokens."""
    case, q = make(dict(n=[40] * 6, lens=[3001] * 6, H=24, HKV=4, D=D, page=64), cache=cache, seed=67)
    mask = mask_of(trees(case.n), 2)
    full, fq = make(dict(n=[64] * 20, lens=[1100] * 20, H=32, HKV=8, D=D, page=64), cache=cache, seed=68)
    fmask = mask_of(trees(full.n), 2)
    caches, scales = case.args()
    fcaches, fscales = full.args()

    def chunk(c, q, caches, scales, most):
        out = torch.zeros(c.T, q.shape[1], D, device="cuda", dtype=torch.bfloat16)
        kda.kda_paged_attention(out, q, *caches, c.cu, c.seq_lens, c.table, most, **scales, check_device=True)
        return out

    want = None
    for amplitude in (1e-3, 1.0, 30.0, 1e3):
        before = (fq.float() * amplitude).to(torch.bfloat16)
        attend(full, before, fmask)
        tree = attend(case, q, mask)[0].clone()
        chunk(full, before, fcaches, fscales, 64)
        line = chunk(case, q, caches, scales, 40)
        want = want or (tree, line)
        assert torch.equal(tree, want[0]) and torch.equal(line, want[1]), f"after queries of {amplitude}"


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_of_padding_tokens_have_no_influence(D, cache):
    """Tokens before position 0 hold anything: huge numbers, infinities, NaN.  Their rows stand in the same warps as those of
    nodes that see something."""
    case, q = make(dict(n=[4, 6, 40], lens=[2, 0, 33], H=12, HKV=2, D=D, page=16), cache=cache, seed=69)
    mask = mask_of(trees(case.n, seed=2), 2)
    q = q.contiguous()
    want, wlse, _ = attend(case, q, mask)
    at = cumulative(case.n)
    for junk in (3e38, float("inf"), float("nan")):
        for b in range(case.B):
            q[at[b]:at[b] + max(0, case.n[b] - case.lens[b])] = junk
        out, lse, status = attend(case, q, mask)
        assert status == 0 and torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_millions_of_requests_without_nodes(cache):
    """Between two that have some: no warp may give up on a note while they are passed over."""
    B, page = 6_000_001, 16
    case, q = make(dict(n=[5, 40], lens=[150, 300], H=12, HKV=2, D=128, page=page), cache=cache, seed=70)
    mask = mask_of(trees(case.n), 2)
    want, wlse, _ = attend(case, q, mask)
    at = torch.zeros(B, dtype=torch.int64, device="cuda")
    at[-1] = 1
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    n[0], n[-1] = case.n
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), n.cumsum(0).to(torch.int32)])
    lens = torch.where(n > 0, case.seq_lens[at], 0)
    table = case.table[at].contiguous()
    out, lse = torch.zeros_like(want), torch.zeros_like(wlse)
    caches, scales = case.args()
    status = kda.kda_tree_attention(out, q, *caches, cu, lens, table, mask, 40, **scales, lse=lse)
    assert int(status.item()) == 0 and torch.equal(out, want) and torch.equal(lse, wlse)
