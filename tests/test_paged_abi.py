"""Refusals of the paged-cache, attention and draft-verification calls: every call
here returns from host validation, before any launch (no GPU needed)."""
import pytest
import torch

import kda_decode_recurrence_gb300 as kda
from kda_decode_recurrence_gb300 import _lib, build

OK, NULL, SHAPE, UNSUP, ENUM, ALIGN, VALUE, WORKSPACE = 0, -1, -2, -3, -4, -6, -7, -8
P = 0x10000  # a fake, aligned address: validation never dereferences


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def args(base, kw):
    unknown = set(kw) - set(base)
    assert not unknown, unknown
    return list({**base, **kw}.values())


CACHE = dict(cache_dtype=1, B=2, T=5, HKV=2, D=128, page_size=64, num_pages=9, max_pages=4)
APPEND = dict(k_cache=P, v_cache=P, k_scale=P, v_scale=P, k=P, v=P, cu=P, lens=P, table=P, **CACHE,
              k_stride=256, v_stride=256, status=None, stream=None)
READ = dict(k_rows=P, v_rows=P, k_cache=P, v_cache=P, k_scale=P, v_scale=P, cu=P, starts=P, table=P,
            **CACHE, status=None, stream=None)
ATTEND = dict(out=P, lse=P, q=P, k_cache=P, v_cache=P, k_scale=P, v_scale=P, cu=P, lens=P, table=P,
              scale=0.1, causal=1, window=0, cache_dtype=1, B=2, T=5, max_tokens=4, H=4, HKV=2, D=128,
              page_size=64, num_pages=9, max_pages=4, q_stride=512, workspace=P,
              workspace_bytes=1 << 40, status=None, stream=None)
VERIFY = dict(tokens=P, accepted=P, target=P, draft=P, draft_tokens=P, accept_u=P, sample_u=P, cu=P,
              B=2, N=3, V=100, target_stride=100, draft_stride=100, status=None, stream=None)

EVERY_CACHE_CALL = [
    ({"B": -1}, SHAPE), ({"T": -1}, SHAPE), ({"HKV": 0}, SHAPE), ({"num_pages": 0}, SHAPE),
    ({"max_pages": 0}, SHAPE), ({"page_size": 0}, SHAPE), ({"D": 0}, SHAPE),
    ({"cache_dtype": 2}, ENUM), ({"cache_dtype": -1}, ENUM),
    ({"D": 96}, UNSUP), ({"D": 256}, UNSUP), ({"page_size": 24}, UNSUP), ({"page_size": 256}, UNSUP),
    ({"page_size": 128, "max_pages": 1 << 24}, UNSUP), ({"num_pages": 1 << 25}, UNSUP),
    ({"k_cache": None}, NULL), ({"v_scale": None}, NULL), ({"table": None}, NULL), ({"cu": None}, NULL),
    ({"k_cache": P + 8}, ALIGN), ({"v_cache": P + 4}, ALIGN), ({"table": P + 2}, ALIGN),
    ({"k_scale": P + 1}, ALIGN), ({"B": 0}, OK), ({"T": 0}, OK),
    ({"T": 0, "k_cache": None, "cu": None}, OK),
]


@pytest.mark.parametrize("kw,expect", EVERY_CACHE_CALL + [
    ({"k_stride": 255}, SHAPE), ({"v_stride": 260}, ALIGN), ({"k": None}, NULL), ({"lens": None}, NULL),
    ({"v": P + 8}, ALIGN), ({"cache_dtype": 0, "k_scale": None, "v_scale": None, "T": 0}, OK)])
def test_append(lib, kw, expect):
    assert lib.kda_cache_append(*args(APPEND, kw)) == expect


@pytest.mark.parametrize("kw,expect", EVERY_CACHE_CALL + [
    ({"k_rows": None}, NULL), ({"v_rows": P + 8}, ALIGN), ({"starts": None, "T": 0}, OK)])
def test_read(lib, kw, expect):
    assert lib.kda_cache_read(*args(READ, kw)) == expect


@pytest.mark.parametrize("kw,expect", EVERY_CACHE_CALL + [
    ({"H": 3}, SHAPE), ({"H": 0}, SHAPE), ({"max_tokens": -1}, SHAPE), ({"q_stride": 504}, SHAPE),
    ({"H": 258, "q_stride": 258 * 128}, UNSUP), ({"T": 1 << 29, "HKV": 1, "H": 4}, UNSUP),
    ({"scale": float("nan")}, VALUE), ({"scale": float("inf")}, VALUE), ({"window": -1}, VALUE),
    ({"causal": 2}, VALUE), ({"out": None}, NULL), ({"q": None}, NULL), ({"lens": None}, NULL),
    ({"q_stride": 516}, ALIGN), ({"out": P + 8}, ALIGN), ({"q": P + 2}, ALIGN), ({"lse": P + 2}, ALIGN),
    ({"workspace": None}, WORKSPACE), ({"workspace_bytes": 16}, WORKSPACE), ({"workspace": P + 128}, ALIGN)])
def test_attention(lib, kw, expect):
    assert lib.kda_paged_attention(*args(ATTEND, kw)) == expect


def test_attention_workspace_size(lib):
    size = lib.kda_paged_attention_workspace_size
    assert size(2, 5, 4, 4, 2, 128) > 0
    for bad in ((-1, 5, 4, 4, 2, 128), (2, -1, 4, 4, 2, 128), (2, 5, -1, 4, 2, 128), (2, 5, 4, 3, 2, 128),
                (2, 5, 4, 4, 0, 128), (2, 5, 4, 4, 2, 96)):
        assert size(*bad) == 0
    for H, HKV, D in ((32, 8, 128), (96, 8, 128), (16, 16, 64), (128, 1, 64)):
        last = 0
        for n in (1, 2, 4, 5, 8, 16, 17, 64, 100, 1000, 4096):  # a larger call never needs less
            now = size(8, 8 * n, n, H, HKV, D)
            assert now >= last
            last = now


@pytest.mark.parametrize("kw,expect", [
    ({"B": -1}, SHAPE), ({"N": -1}, SHAPE), ({"V": 0}, SHAPE), ({"target_stride": 99}, SHAPE),
    ({"draft_stride": 99}, SHAPE), ({"B": 1 << 29}, UNSUP),
    ({"tokens": None}, NULL), ({"accepted": None}, NULL), ({"target": None}, NULL),
    ({"sample_u": None}, NULL), ({"cu": None}, NULL), ({"draft_tokens": None}, NULL),
    ({"accept_u": None}, NULL), ({"target": P + 2}, ALIGN), ({"tokens": P + 1}, ALIGN),
    ({"B": 0}, OK), ({"B": 0, "draft": None, "draft_stride": 0}, OK)])
def test_verify(lib, kw, expect):
    assert lib.kda_verify_draft(*args(VERIFY, kw)) == expect


def test_binding_refusals():
    """The binding's own checks come before the library is called (CPU tensors)."""
    i32 = dict(dtype=torch.int32)
    k = torch.zeros(9, 2, 64, 128, dtype=torch.bfloat16)
    x = torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    cu, lens, table = torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, 4, **i32)
    good = dict(k_cache=k, v_cache=k, k=x, v=x, cu_seqlens=cu, seq_lens=lens, page_table=table)
    for change, error in [
            (dict(k_cache=k.half(), v_cache=k.half()), TypeError), (dict(v_cache=k[:8]), ValueError),
            (dict(v_cache=k.transpose(1, 2)), ValueError), (dict(k_scale=torch.zeros(9, 2, 64)), ValueError),
            (dict(k=x.float()), TypeError), (dict(k=x[:, :1]), ValueError), (dict(v=x[:4]), ValueError),
            (dict(k=x.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
            (dict(cu_seqlens=cu[:2]), ValueError), (dict(cu_seqlens=cu.long()), TypeError),
            (dict(seq_lens=torch.zeros(3, **i32)), ValueError), (dict(page_table=table[0]), ValueError),
            (dict(k_cache=k.to(torch.float8_e4m3fn), v_cache=k.to(torch.float8_e4m3fn)), ValueError)]:
        with pytest.raises(error):
            kda.kda_cache_append(**{**good, **change})
    out = torch.zeros(5, 4, 128, dtype=torch.bfloat16)
    good = dict(out=out, q=out, k_cache=k, v_cache=k, cu_seqlens=cu, seq_lens=lens, page_table=table, max_tokens=3)
    for change, error in [(dict(out=out.float()), TypeError), (dict(out=out[:4]), ValueError),
                          (dict(q=out[:, :, :64]), ValueError), (dict(lse=torch.zeros(5, 3)), ValueError),
                          (dict(workspace=torch.zeros(8)), TypeError)]:
        with pytest.raises(error):
            kda.kda_paged_attention(**{**good, **change})
    f = torch.zeros
    good = dict(tokens=f(5, **i32), accepted=f(2, **i32), target_probs=f(5, 10), draft_probs=f(3, 10),
                draft_tokens=f(3, **i32), accept_u=f(3), sample_u=f(2), cu_drafts=cu)
    for change, error in [(dict(target_probs=f(5, 10).double()), TypeError), (dict(target_probs=f(4, 10)), ValueError),
                          (dict(draft_probs=f(3, 9)), ValueError), (dict(tokens=f(4, **i32)), ValueError),
                          (dict(target_probs=f(10, 5).t()), ValueError), (dict(accept_u=f(2)), ValueError)]:
        with pytest.raises(error):
            kda.kda_verify_draft(**{**good, **change})


def test_host_tensors_are_refused(lib):
    """Tensors in host memory are refused also where a stream and a status word are given (no
    address of theirs reaches a kernel)."""
    class Stream:
        cuda_stream = 0

    i32 = dict(dtype=torch.int32)
    k = torch.zeros(9, 2, 64, 128, dtype=torch.bfloat16)
    x = torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    cu, lens, table = torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, 4, **i32)
    f, rest = torch.zeros, dict(dev_status=torch.zeros(1, **i32), stream=Stream())
    with pytest.raises(ValueError):
        kda.kda_cache_append(k, k, x, x, cu, lens, table, **rest)
    with pytest.raises(ValueError):
        kda.kda_cache_read(x, x, k, k, cu, None, table, **rest)
    with pytest.raises(ValueError):
        kda.kda_paged_attention(x, x, k, k, cu, lens, table, 3, workspace=f(1 << 25, dtype=torch.uint8), **rest)
    with pytest.raises(ValueError):
        kda.kda_verify_draft(f(5, **i32), f(2, **i32), f(5, 10), f(3, 10), f(3, **i32), f(3), f(2), cu, **rest)
