"""kda_cache_append and kda_cache_read against their formula in 64 bits.

The scales and the codes of kda_cache_append have one right value each (quotients
rounded to nearest in fp32, the code to nearest even), so they are compared for
equality; kda_cache_read is off by one rounding to fp32 and one to bf16."""
import numpy as np
import pytest
import torch

import kda_decode_recurrence_gb300 as kda

from _paged import Case, E4M3_TABLE, U_BF16, U_F32, cumulative, quantise
from _parity import Guarded, guarded_copy

pytestmark = pytest.mark.gpu


def bits(t):
    return t.cpu().view(torch.uint8 if t.element_size() == 1 else torch.int16).numpy()


def append(case, k, v, table=None, seq_lens=None, cu=None):
    """Run kda_cache_append on guarded copies of the cache; returns them and the status."""
    held = {}
    for name in ("k", "v"):
        x, s = case.tensors[name]
        held[name] = guarded_copy(x)
        held[name + "_scale"] = None if s is None else guarded_copy(s)
    scales = {n: None if held[n] is None else held[n].t for n in ("k_scale", "v_scale")}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_cache_append(held["k"].t, held["v"].t, k, v, case.cu if cu is None else cu,
                         case.seq_lens if seq_lens is None else seq_lens,
                         case.table if table is None else table, **scales, dev_status=status)
    torch.cuda.synchronize()
    assert all(g is None or g.intact() for g in held.values())
    return held, int(status.item())


def rows(case, seed, wild=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(case.T, 2, case.HKV, case.D, generator=g)
    x *= torch.exp2(torch.randint(-30, 30, (case.T, 2, case.HKV, 1), generator=g).float())
    x = x.to(torch.bfloat16)
    if wild and case.T >= 8:
        x[0, 0, 0] = 0
        x[1, 1, 0, 3] = float("inf")
        x[2, 0, 0, 5] = float("nan")
        x[3, :, :] = -0.0
        x[4, 0, 0] = torch.finfo(torch.bfloat16).tiny     # scales below the normal range
        x[5, 0, 0, :] = torch.tensor([2.0 ** -133, 0.0]).repeat(case.D // 2)
        x[6, 0, 0] = torch.finfo(torch.bfloat16).max
        x[7, 0, 0] = torch.linspace(-448, 448, case.D)    # ties of the code's rounding
    x = x.cuda()
    return x[:, 0], x[:, 1]                               # tokens strided by 2 HKV D


SHAPES = [
    dict(n=[1], lens=[1], HKV=1, D=128, page=16),
    dict(n=[1, 1, 1], lens=[1, 64, 65], HKV=8, D=128, page=64),
    dict(n=[0, 5, 0, 1, 0], lens=[0, 40, 7, 1, 300], HKV=3, D=64, page=16),
    dict(n=[33, 17, 129], lens=[33, 150, 129], HKV=2, D=128, page=32),
    dict(n=[300], lens=[300], HKV=1, D=64, page=128),
    dict(n=[4, 9], lens=[2, 8], HKV=2, D=128, page=16),   # tokens before position 0
    dict(n=list(range(40)), lens=[2 * i for i in range(40)], HKV=2, D=128, page=16),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=range(len(SHAPES)))
def test_append(shape, cache):
    case = Case(**shape, cache=cache, seed=3, junk=1.0)
    k, v = rows(case, 5, wild=True)
    held, status = append(case, k, v)
    assert status == 0
    for name, x in (("k", k), ("v", v)):
        before, scale0 = case.tensors[name]
        want = bits(before).copy()
        codes, scales = quantise(x.float().cpu().numpy()) if cache == "e4m3" else (bits(x.contiguous()), None)
        want_scale = None if scale0 is None else scale0.cpu().numpy().copy()
        cu = cumulative(case.n)
        for b in range(case.B):
            for i in range(case.n[b]):
                pos = case.lens[b] - case.n[b] + i
                if pos < 0:
                    continue
                pg, off = int(case.table[b, pos // case.page]), pos % case.page
                for h in range(case.HKV):
                    nan = scales is not None and np.isnan(scales[cu[b] + i, h])
                    want[pg, h, off] = bits(held[name].t)[pg, h, off] if nan else codes[cu[b] + i, h]
                    if scales is not None:
                        want_scale[pg, h, off] = scales[cu[b] + i, h]
        assert np.array_equal(bits(held[name].t), want), name
        if scales is not None:
            assert np.array_equal(held[name + "_scale"].t.cpu().numpy(), want_scale, equal_nan=True), name


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=range(len(SHAPES)))
@pytest.mark.parametrize("from_start", [True, False])
def test_read(shape, cache, from_start):
    case = Case(**shape, cache=cache, seed=4)
    lens = [max(x, 0) for x in case.lens]
    starts = [0] * case.B if from_start else [x // 3 for x in lens]
    n = [x - s for x, s in zip(lens, starts)]
    cu = torch.tensor(cumulative(n), dtype=torch.int32, device="cuda")
    outs = [Guarded((sum(n), case.HKV, case.D), torch.bfloat16, fill=float("nan")) for _ in range(2)]
    caches, scales = case.args()
    status = kda.kda_cache_read(outs[0].t, outs[1].t, *caches, cu,
                                None if from_start else torch.tensor(starts, dtype=torch.int32, device="cuda"),
                                case.table, **scales)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and all(o.intact() for o in outs)
    for name, o in zip(("k", "v"), outs):
        want = torch.cat([case.dense(name, b)[starts[b]:] for b in range(case.B)])
        off = (o.t.double() - want).abs()
        assert bool((off <= (U_BF16 + 2 * U_F32) * want.abs() if cache == "e4m3" else off == 0).all())


def test_every_quotient_of_two_bf16_fractions():
    """Codes depend on the fractions of an entry and of its row's largest and on how far
    apart their exponents are: all 128 x 128 x 20 of them, compared for equality."""
    most = torch.arange(128) * 2.0 ** -7 + 1                       # the row's largest entry
    part = (torch.arange(128) * 2.0 ** -7 + 1)[None] * torch.exp2(-torch.arange(20.0))[:, None]
    part = part.flatten()
    x = torch.zeros(128, 21, 128)                                   # 20 rows of 127 entries and some
    entries = torch.minimum(part[None].expand(128, -1), most[:, None])
    x.view(128, -1)[:, :entries.shape[1]] = entries
    x[:, :, 127] = most[:, None]
    x.view(128, -1)[:, entries.shape[1]:entries.shape[1] + 20] = entries[:, 127::128]   # those that 127 took
    x = x.reshape(-1, 1, 128).to(torch.bfloat16)
    case = Case(n=[len(x)], lens=[len(x)], HKV=1, D=128, page=128, cache="e4m3", junk=0.0)
    held, status = append(case, x.cuda(), -x.cuda())
    assert status == 0
    codes, scales = quantise(x.float().numpy())
    pages = case.table[0, :-(-len(x) // 128)].long()
    for name, sign in (("k", 0), ("v", 0x80)):
        got = bits(held[name].t[pages])[:, 0].reshape(-1, 128)[:len(x)]
        assert np.array_equal(got, codes[:, 0] ^ sign)
        assert np.array_equal(held[name + "_scale"].t[pages].cpu().numpy()[:, 0].reshape(-1)[:len(x)], scales[:, 0])


def test_round_trip_is_within_half_a_step():
    case = Case(n=[500], lens=[500], HKV=4, D=128, page=64, cache="e4m3", seed=6)
    k, v = rows(case, 7)
    held, status = append(case, k, v)
    assert status == 0
    out = [torch.empty(500, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kda.kda_cache_read(*out, held["k"].t, held["v"].t, case.cu, None, case.table,
                       k_scale=held["k_scale"].t, v_scale=held["v_scale"].t)
    for x, y in ((k, out[0]), (v, out[1])):
        x, y = x.double(), y.double()
        scale = x.abs().amax(-1, keepdim=True) / 448
        # e4m3 2^-4 of the value, half the smallest step 2^-10 of the scale; bf16 on top
        bound = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * scale) * (1 + 1e-5) + U_BF16 * y.abs()
        assert bool(((x - y).abs() <= bound).all())


def test_a_row_that_is_not_finite_reads_back_as_nan():
    case = Case(n=[9], lens=[9], HKV=1, D=64, page=16, cache="e4m3", junk=0.0)
    k, v = rows(case, 5, wild=True)
    held, _ = append(case, k, v)
    out = [torch.empty(9, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kda.kda_cache_read(*out, held["k"].t, held["v"].t, case.cu, None, case.table,
                       k_scale=held["k_scale"].t, v_scale=held["v_scale"].t)
    for x, y in ((k, out[0]), (v, out[1])):
        bad = ~torch.isfinite(x).all(-1)
        assert int(bad.sum()) == 1
        assert bool(torch.isnan(y[bad]).all()) and bool(torch.isfinite(y[~bad]).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_bad_pages_and_lengths_are_reported_and_skipped(cache):
    shape = dict(n=[3, 4, 5], lens=[20, 40, 30], HKV=2, D=128, page=16)
    case = Case(**shape, cache=cache, junk=1.0)
    k, v = rows(case, 9)
    good, status = append(case, k, v)
    assert status == 0
    table = case.table.clone()
    table[1, 2] = case.num_pages                       # request 1's new tokens: positions 36..39
    held, status = append(case, k, v, table=table)
    assert status == kda.DEV_BAD_PAGE
    mine = int(case.table[1, 2])
    for name in ("k", "v"):
        want = good[name].t.clone()
        want.view(torch.uint8)[mine] = case.tensors[name][0].view(torch.uint8)[mine]
        assert np.array_equal(bits(held[name].t), bits(want))
    lens = torch.tensor([20, case.max_pages * 16 + 1, -1], dtype=torch.int32, device="cuda")
    held, status = append(case, k, v, seq_lens=lens)   # requests 1 and 2 are skipped
    assert status == kda.DEV_BAD_SEQLEN
    cu = torch.tensor([0, 3, 7, 999], dtype=torch.int32, device="cuda")
    _, status = append(case, k, v, cu=cu)
    assert status == kda.DEV_BAD_SEQLEN
    caches, scales = case.args()
    out = [torch.full((12, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    starts = torch.tensor([17, 36, 25], dtype=torch.int32, device="cuda")
    status = kda.kda_cache_read(*out, *caches, case.cu, starts, table, **scales)
    assert int(status.item()) == kda.DEV_BAD_PAGE
    assert all(bool((o[3:7] == 0).all()) and bool((o[7:] != 0).any()) for o in out)
    starts[0] = case.max_pages * 16 - 2                # its third row is past the table's end
    status = kda.kda_cache_read(*out, *caches, case.cu, starts, case.table, **scales)
    assert int(status.item()) == kda.DEV_BAD_SEQLEN and all(bool((o[:3] == 0).all()) for o in out)


def test_offsets_beyond_32_bits():
    """A cache of 2.4e9 entries: the last page's rows lie past 2^31 elements and 2^32 bytes."""
    pages, HKV, D, page = 18400, 8, 128, 128
    k = torch.zeros(pages, HKV, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 130], dtype=torch.int32, device="cuda")
    lens = torch.tensor([130], dtype=torch.int32, device="cuda")
    x = torch.randn(130, HKV, D, device="cuda").to(torch.bfloat16)
    assert int(kda.kda_cache_append(k, v, x, -x, cu, lens, table).item()) == 0
    assert torch.equal(k[-1], x[:128].transpose(0, 1)) and torch.equal(v[0, :, :2], -x[128:].transpose(0, 1))
    assert int((k != 0).any(-1).sum()) == 130 * HKV
    out = [torch.empty_like(x) for _ in range(2)]
    assert int(kda.kda_cache_read(*out, k, v, cu, None, table).item()) == 0
    assert torch.equal(out[0], x) and torch.equal(out[1], -x)


def test_table_of_code_values():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(codes.float().numpy().astype(np.float64), E4M3_TABLE, equal_nan=True)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_every_malformed_request_is_reported(cache):
    """Also where no row of the call shows it: offsets that start past 0 or before it, end
    before T or past it, or go back; a bad length of a request without new rows."""
    case = Case(n=[3, 0, 5], lens=[20, 12, 30], HKV=2, D=64, page=16, cache=cache, junk=1.0)
    k, v = rows(case, 9)
    good, status = append(case, k, v)
    assert status == 0
    caches, scales = case.args()
    out = [torch.zeros(case.T, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    i32 = dict(dtype=torch.int32, device="cuda")
    starts = case.seq_lens - torch.tensor(case.n, **i32)
    assert int(kda.kda_cache_read(*out, *caches, case.cu, starts, case.table, **scales)) == 0
    # the last three leave every row of the call in a well-formed request
    for cu in ([1, 3, 3, 8], [0, 3, 3, 7], [0, 3, 3, 9], [-2, 3, 3, 8], [0, 8, 3, 8], [0, 8, 8, 7], [-1, 0, 0, 8]):
        cu = torch.tensor(cu, **i32)
        _, status = append(case, k, v, cu=cu, seq_lens=torch.full((3,), 30, **i32))
        assert status == kda.DEV_BAD_SEQLEN, cu
        assert int(kda.kda_cache_read(*out, *caches, cu, None, case.table, **scales)) == kda.DEV_BAD_SEQLEN, cu
    for bad in (-1, case.max_pages * 16 + 1):
        lens = case.seq_lens.clone()
        lens[1] = bad                                       # request 1 has no new rows
        held, status = append(case, k, v, seq_lens=lens)
        assert status == kda.DEV_BAD_SEQLEN
        for name in ("k", "v"):                             # and the others are served
            assert np.array_equal(bits(held[name].t), bits(good[name].t))
        starts[1] = bad
        assert int(kda.kda_cache_read(*out, *caches, case.cu, starts, case.table, **scales)) == kda.DEV_BAD_SEQLEN


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,HKV,D,page", [(38912, 1, 64, 128), (45001, 3, 128, 64), (100003, 2, 64, 16), (170001, 1, 128, 32)])
def test_many_rows(T, HKV, D, page, cache):
    """Calls in which a warp takes two tokens and more (from 2 x 152 x 128 on): every row of
    ragged requests, some with padding, is in its place and reads back."""
    cut = sorted(np.random.default_rng(T).integers(0, T, 9).tolist())
    n = np.diff([0] + cut + [T]).tolist()
    lens = [x + 5 * i for i, x in enumerate(n)]
    lens[3] = max(0, n[3] - 2)                                  # two tokens of padding
    need = [-(-x // page) for x in lens]
    g = torch.Generator(device="cuda").manual_seed(T)
    pages, width = sum(need) + 1, max(need) + 1
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(n), width), -1, dtype=torch.int32, device="cuda")
    for b, at in enumerate(cumulative(need)[:-1]):
        table[b, :need[b]] = order[at:at + need[b]]
    x = torch.randn(T, 2, HKV, D, device="cuda", generator=g).to(torch.bfloat16)
    dtype = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    kc, vc = [torch.zeros(pages, HKV, page, D, device="cuda").to(dtype) for _ in range(2)]
    scales = {} if cache == "bf16" else {s: torch.zeros(pages, HKV, page, device="cuda") for s in ("k_scale", "v_scale")}
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, seq = torch.tensor(cumulative(n), **i32), torch.tensor(lens, **i32)
    assert int(kda.kda_cache_append(kc, vc, x[:, 0], x[:, 1], cu, seq, table, **scales)) == 0
    b = torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"))
    pos = seq.long()[b] - cu.long()[b + 1] + torch.arange(T, device="cuda")
    real = pos >= 0
    row = (table[b, pos.clamp_min(0) // page].long() * page + pos.clamp_min(0) % page)[real]   # place among all pages' rows
    for c, s, y in ((kc, scales.get("k_scale"), x[:, 0]), (vc, scales.get("v_scale"), x[:, 1])):
        got = c.view(torch.uint8).transpose(1, 2).reshape(pages * page, HKV, -1)
        y = y[real].contiguous()
        if s is None:
            codes = y.view(torch.uint8).reshape(got[row].shape)
        else:
            code, scale = quantise(y.float().cpu().numpy())
            codes = torch.from_numpy(code).cuda()
            assert torch.equal(s.transpose(1, 2).reshape(pages * page, HKV)[row], torch.from_numpy(scale).cuda())
        assert torch.equal(got[row], codes)
        rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        rest[row] = False
        assert not bool(got[rest].any())
    out = [torch.full((T, HKV, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    starts = torch.tensor([L - m for L, m in zip(lens, n)], **i32)
    starts[3] = 0                                               # its rows 0 .. lens, then two without a page in use
    if need[3] * page < n[3]:
        table[3, need[3]] = table[3, need[3] - 1]
    assert int(kda.kda_cache_read(*out, kc, vc, cu, starts, table, **scales)) == 0
    place = torch.arange(T, device="cuda") - cu.long()[b] + starts.long()[b]
    at = table[b, place // page].long() * page + place % page
    for c, s, y in ((kc, scales.get("k_scale"), out[0]), (vc, scales.get("v_scale"), out[1])):
        flat = c.transpose(1, 2).reshape(pages * page, HKV, D)
        want = flat.view(torch.uint8)[at].view(c.dtype).float() if s is not None else flat[at].float()
        if s is not None:
            want = (want * s.transpose(1, 2).reshape(pages * page, HKV)[at][..., None]).to(torch.bfloat16).float()
        assert torch.equal(y.float(), want)
