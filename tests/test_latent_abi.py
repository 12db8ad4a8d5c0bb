"""Refusals of the latent-cache, latent-attention and tree-attention calls: every call here returns
from host validation, before any launch (no GPU needed)."""
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


APPEND = dict(cache=P, rows=P, gamma=P, eps=1e-5, cu=P, lens=P, table=P, B=2, T=5, page_size=64, num_pages=9,
              max_pages=4, stride=576, status=None, stream=None)
ATTEND = dict(out=P, lse=P, q=P, cache=P, cu=P, lens=P, table=P, mask=P, scale=0.1, causal=1, B=2, T=5, H=4,
              mask_words=1, page_size=64, num_pages=9, max_pages=4, q_stride=4 * 576, workspace=P,
              workspace_bytes=1 << 40, status=None, stream=None)
EXPANDED = dict(out=P, lse=P, q=P, kv=P, k_pe=P, cu_q=P, cu_k=P, scale=0.1, causal=1, B=2, Tq=5, Tk=9, H=4,
                q_stride=4 * 192, kv_stride=4 * 256, pe_stride=64, workspace=P, workspace_bytes=1 << 40, status=None,
                stream=None)
TREE = dict(out=P, lse=P, q=P, k_cache=P, v_cache=P, k_scale=P, v_scale=P, cu=P, lens=P, table=P, mask=P, scale=0.1,
            cache_dtype=1, B=2, T=5, max_tokens=4, mask_words=1, H=4, HKV=2, D=128, page_size=64, num_pages=9,
            max_pages=4, q_stride=512, workspace=P, workspace_bytes=1 << 40, status=None, stream=None)

LATENT_CALL = [
    ({"B": -1}, SHAPE), ({"T": -1}, SHAPE), ({"page_size": 0}, SHAPE), ({"num_pages": 0}, SHAPE),
    ({"max_pages": 0}, SHAPE), ({"page_size": 24}, UNSUP), ({"page_size": 256}, UNSUP),
    ({"page_size": 128, "max_pages": 1 << 24}, UNSUP), ({"num_pages": 1 << 25}, UNSUP),
    ({"cache": None}, NULL), ({"table": None}, NULL), ({"cu": None}, NULL), ({"lens": None}, NULL),
    ({"cache": P + 8}, ALIGN), ({"table": P + 2}, ALIGN), ({"cu": P + 1}, ALIGN), ({"lens": P + 2}, ALIGN),
    ({"B": 0}, OK), ({"T": 0}, OK), ({"T": 0, "cache": None, "cu": None}, OK)]


@pytest.mark.parametrize("kw,expect", LATENT_CALL + [
    ({"rows": None}, NULL), ({"rows": P + 8}, ALIGN), ({"gamma": P + 4}, ALIGN), ({"gamma": None, "T": 0}, OK),
    ({"stride": 575}, SHAPE), ({"stride": 580}, ALIGN), ({"eps": -1e-6}, VALUE), ({"eps": float("nan")}, VALUE),
    ({"eps": float("inf")}, VALUE)])
def test_append(lib, kw, expect):
    assert lib.kda_latent_append(*args(APPEND, kw)) == expect


@pytest.mark.parametrize("kw,expect", LATENT_CALL + [
    ({"H": 0}, SHAPE), ({"q_stride": 4 * 576 - 8}, SHAPE), ({"mask_words": 0}, SHAPE), ({"mask_words": -1}, SHAPE),
    ({"T": 1 << 28}, UNSUP), ({"mask_words": 1 << 25}, UNSUP), ({"scale": float("nan")}, VALUE),
    ({"scale": float("-inf")}, VALUE), ({"causal": 2}, VALUE), ({"causal": -1}, VALUE), ({"out": None}, NULL),
    ({"q": None}, NULL), ({"q_stride": 4 * 576 + 4}, ALIGN), ({"out": P + 8}, ALIGN), ({"q": P + 2}, ALIGN),
    ({"lse": P + 2}, ALIGN), ({"mask": P + 2}, ALIGN), ({"workspace": None}, WORKSPACE),
    ({"workspace_bytes": 16}, WORKSPACE), ({"workspace": P + 128}, ALIGN)])
def test_attention(lib, kw, expect):
    assert lib.kda_latent_attention(*args(ATTEND, kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"B": -1}, SHAPE), ({"Tq": -1}, SHAPE), ({"Tk": -1}, SHAPE), ({"H": 0}, SHAPE), ({"q_stride": 760}, SHAPE),
    ({"kv_stride": 1016}, SHAPE), ({"pe_stride": 56}, SHAPE), ({"Tq": 1 << 28}, UNSUP), ({"Tk": (1 << 30) + 1}, UNSUP),
    ({"scale": float("nan")}, VALUE), ({"scale": float("inf")}, VALUE), ({"causal": 2}, VALUE), ({"out": None}, NULL),
    ({"q": None}, NULL), ({"kv": None}, NULL), ({"k_pe": None}, NULL), ({"cu_q": None}, NULL), ({"cu_k": None}, NULL),
    ({"out": P + 8}, ALIGN), ({"q": P + 2}, ALIGN), ({"kv": P + 8}, ALIGN), ({"k_pe": P + 8}, ALIGN), ({"lse": P + 2}, ALIGN),
    ({"q_stride": 772}, ALIGN), ({"kv_stride": 1028}, ALIGN), ({"pe_stride": 68}, ALIGN), ({"cu_q": P + 1}, ALIGN),
    ({"cu_k": P + 2}, ALIGN), ({"workspace": None}, WORKSPACE), ({"workspace_bytes": 16}, WORKSPACE),
    ({"workspace": P + 128}, ALIGN), ({"B": 0}, OK), ({"Tq": 0}, OK), ({"Tq": 0, "q": None, "cu_q": None}, OK)])
def test_expanded(lib, kw, expect):
    assert lib.kda_latent_expanded(*args(EXPANDED, kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"B": -1}, SHAPE), ({"HKV": 0}, SHAPE), ({"cache_dtype": 2}, ENUM), ({"D": 96}, UNSUP), ({"page_size": 24}, UNSUP),
    ({"k_cache": None}, NULL), ({"v_scale": None}, NULL), ({"table": None}, NULL), ({"cu": None}, NULL),
    ({"lens": None}, NULL), ({"mask": None}, NULL), ({"out": None}, NULL), ({"q": None}, NULL),
    ({"H": 3}, SHAPE), ({"max_tokens": -1}, SHAPE), ({"max_tokens": 33}, SHAPE), ({"mask_words": 0}, SHAPE),
    ({"q_stride": 504}, SHAPE), ({"H": 258, "q_stride": 258 * 128}, UNSUP), ({"scale": float("nan")}, VALUE),
    ({"mask": P + 2}, ALIGN), ({"q_stride": 516}, ALIGN), ({"out": P + 8}, ALIGN), ({"workspace": None}, WORKSPACE),
    ({"workspace_bytes": 16}, WORKSPACE), ({"workspace": P + 128}, ALIGN), ({"B": 0}, OK), ({"T": 0}, OK)])
def test_tree(lib, kw, expect):
    assert lib.kda_tree_attention(*args(TREE, kw)) == expect


def test_workspace_sizes(lib):
    size = lib.kda_tree_attention_workspace_size
    assert size(2, 5, 4, 4, 2, 128) > 0
    for bad in ((-1, 5, 4, 4, 2, 128), (2, -1, 4, 4, 2, 128), (2, 5, -1, 4, 2, 128), (2, 5, 4, 3, 2, 128),
                (2, 5, 4, 4, 2, 96)):
        assert size(*bad) == 0
    size = lib.kda_latent_expanded_workspace_size
    assert size(2, 5, 4) > 0 and size(1000, 5000, 128) >= size(2, 5, 4)
    for bad in ((-1, 5, 4), (2, -1, 4), (2, 5, 0)):
        assert size(*bad) == 0
    size = lib.kda_latent_attention_workspace_size
    assert size(2, 5, 4) > 0 and size(1000, 5000, 128) >= size(2, 5, 4)
    for bad in ((-1, 5, 4), (2, -1, 4), (2, 5, 0)):
        assert size(*bad) == 0


def test_binding_refusals(lib):
    """The binding's own checks come before the library is called; tensors in host memory are
    refused also where a stream and a status word are given."""
    class Stream:
        cuda_stream = 0

    i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    cache, rows = torch.zeros(9, 64, 576, **bf), torch.zeros(5, 576, **bf)
    cu, lens, table = torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, 4, **i32)
    rest = dict(dev_status=torch.zeros(1, **i32), stream=Stream())
    good = dict(cache=cache, rows=rows, cu_seqlens=cu, seq_lens=lens, page_table=table, **rest)
    for change, error in [
            (dict(), ValueError), (dict(cache=cache.half()), TypeError), (dict(cache=cache[:, :, :512]), ValueError),
            (dict(cache=cache[0]), ValueError), (dict(rows=rows.float()), TypeError), (dict(rows=rows[:, :500]), ValueError),
            (dict(rows=rows[0]), ValueError), (dict(gamma=torch.zeros(511)), ValueError),
            (dict(gamma=torch.zeros(512, **bf)), TypeError), (dict(cu_seqlens=cu[:2]), ValueError),
            (dict(cu_seqlens=cu.long()), TypeError), (dict(seq_lens=lens[:1]), ValueError), (dict(page_table=table[0]), ValueError)]:
        with pytest.raises(error):
            kda.kda_latent_append(**{**good, **change})
    out, q, mask = torch.zeros(5, 4, 512, **bf), torch.zeros(5, 4, 576, **bf), torch.zeros(5, 1, **i32)
    good = dict(out=out, q=q, cache=cache, cu_seqlens=cu, seq_lens=lens, page_table=table,
                workspace=torch.zeros(1 << 20, dtype=torch.uint8), **rest)
    for change, error in [
            (dict(), ValueError), (dict(out=out.float()), TypeError), (dict(out=out[:4]), ValueError),
            (dict(out=torch.zeros(5, 4, 576, **bf)), ValueError), (dict(q=q[:, :, :512]), ValueError), (dict(q=q[0]), ValueError),
            (dict(lse=torch.zeros(5, 3)), ValueError), (dict(lse=torch.zeros(5, 4).double()), TypeError),
            (dict(tree_mask=mask[:4]), ValueError), (dict(tree_mask=mask[:, 0]), ValueError), (dict(tree_mask=mask.long()), TypeError)]:
        with pytest.raises(error):
            kda.kda_latent_attention(**{**good, **change})
    k, x = torch.zeros(9, 2, 64, 128, **bf), torch.zeros(5, 4, 128, **bf)
    qe, kv, pe = torch.zeros(5, 4, 192, **bf), torch.zeros(9, 4, 256, **bf), torch.zeros(9, 64, **bf)
    good = dict(out=x, q=qe, kv=kv, k_pe=pe, cu_q=cu, cu_k=cu, workspace=torch.zeros(1 << 20, dtype=torch.uint8), **rest)
    for change, error in [
            (dict(), ValueError), (dict(q=qe.float()), TypeError), (dict(q=qe[:, :, :128]), ValueError), (dict(q=qe[0]), ValueError),
            (dict(kv=kv[:, :3]), ValueError), (dict(kv=kv.half()), TypeError), (dict(k_pe=pe[:8]), ValueError),
            (dict(k_pe=pe[:, :32]), ValueError), (dict(k_pe=pe.t().contiguous().t()), ValueError), (dict(out=x[:4]), ValueError),
            (dict(cu_k=cu[:2]), ValueError), (dict(cu_q=cu.long()), TypeError), (dict(lse=torch.zeros(5, 3)), ValueError),
            (dict(cu_q=cu[:0], cu_k=cu[:0]), ValueError)]:
        with pytest.raises(error):
            kda.kda_latent_expanded(**{**good, **change})
    good = dict(out=x, q=x, k_cache=k, v_cache=k, cu_seqlens=cu, seq_lens=lens, page_table=table, tree_mask=mask,
                max_tokens=3, workspace=torch.zeros(1 << 20, dtype=torch.uint8), **rest)
    for change, error in [
            (dict(), ValueError), (dict(tree_mask=mask[:4]), ValueError), (dict(tree_mask=mask.float()), TypeError),
            (dict(out=x[:4]), ValueError), (dict(q=x[:, :3]), ValueError), (dict(seq_lens=lens[:1]), ValueError),
            (dict(lse=torch.zeros(5, 3)), ValueError)]:
        with pytest.raises(error):
            kda.kda_tree_attention(**{**good, **change})
