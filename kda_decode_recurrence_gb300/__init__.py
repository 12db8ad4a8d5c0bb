"""GB300-native KDA token-generation library: Python binding of libkda.

The functions are the C-ABI calls of include/kda.h, under the same names;
this module only checks tensors and marshals their device pointers, sizes and
the current CUDA stream.  Every step of the computation runs in libkda's CUDA
kernels; there is no CPU or PyTorch fallback, and a missing library raises.

Each call returns its device status word (an int32 CUDA tensor: KDA_DEV_*
bits the kernels OR in).  Pass ``dev_status`` to reuse one; when none is
passed, a zeroed word is allocated on the call's stream, so that device-side
reports (a bad slot, a malformed cu_seqlens, a pipeline timeout) are never
dropped.  ``check_device=True`` synchronises the stream and raises
KdaDeviceError when any bit is set.

    kda_decode(output, q, k, v, raw_gate, beta_logits, a_log, dt_bias,
               cu_seqlens, state_pool, state_indices, gate_mode, lower_bound)
    kda_decode_ex(..., state_layout=STATE_K_FIRST | STATE_V_FIRST)
               (the output dtype, fp32 or bf16, is taken from `output`)
    kda_prefill(<the arguments of kda_decode>)   16-token chunks
    kda_block_tkg(out, hidden, gamma_in, W_in, W_fb, W_gb, conv_w, A_log,
                  dt_bias, gamma_o, W_o, S, conv_state, scale, lower_bound,
                  rms_norm_eps, l2_eps, workspace)
    block_workspace_size(B, n, Hd, nh, K, V, Kc)

Next to the KDA layers, for a model's full-attention layers and drafted tokens:

    kda_cache_append(k_cache, v_cache, k, v, cu_seqlens, seq_lens, page_table)
    kda_cache_read(k_rows, v_rows, k_cache, v_cache, cu_rows, starts, page_table)
    kda_paged_attention(out, q, k_cache, v_cache, cu_seqlens, seq_lens,
                        page_table, max_tokens)
    paged_attention_workspace_size(B, T, max_tokens, H, HKV, D)
    kda_verify_draft(tokens, accepted, target_probs, draft_probs, draft_tokens,
                     accept_u, sample_u, cu_drafts)
"""
from __future__ import annotations

import torch

from . import _lib

GATE_SOFTPLUS = 0
GATE_LOWER_BOUND = 1
STATE_K_FIRST = 0
STATE_V_FIRST = 1
OUTPUT_F32 = 0
OUTPUT_BF16 = 1
DEV_BAD_SLOT = 1
DEV_BAD_SEQLEN = 2
DEV_TIMEOUT = 4
DEV_BOUNDS = 8  # debug builds only (libkda_debugbounds.so)
DEV_BAD_PAGE = 16
DEV_BAD_TOKEN = 32
DEV_BAD_PROB = 64
CACHE_BF16 = 0
CACHE_E4M3 = 1


class KdaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        name = _lib.STATUS.get(status, str(status))
        super().__init__(f"{what} failed: {name} ({_lib.load().kda_status_string(status).decode()})")


class KdaDeviceError(RuntimeError):
    def __init__(self, bits: int, what: str):
        self.bits = bits
        names = [n for b, n in ((DEV_BAD_SLOT, "KDA_DEV_BAD_SLOT"),
                                (DEV_BAD_SEQLEN, "KDA_DEV_BAD_SEQLEN"),
                                (DEV_TIMEOUT, "KDA_DEV_TIMEOUT"),
                                (DEV_BOUNDS, "KDA_DEV_BOUNDS"),
                                (DEV_BAD_PAGE, "KDA_DEV_BAD_PAGE"),
                                (DEV_BAD_TOKEN, "KDA_DEV_BAD_TOKEN"),
                                (DEV_BAD_PROB, "KDA_DEV_BAD_PROB")) if bits & b]
        super().__init__(f"{what}: device status {bits} ({' | '.join(names) or 'unknown bits'})")


def _check(t: torch.Tensor, name: str, dtype, device) -> None:
    if t.dtype is dtype and t.device == device and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _stream_of(stream, device) -> int:
    """The handle of the caller's stream, or of the current one of ``device`` (by the raw
    handle: the small calls take less time than building a Stream object).  Host tensors,
    whose device has no index, are refused (its ``type`` is a string made at each look: 0.7 us)."""
    index = device.index
    if index is None:
        raise ValueError(f"expected CUDA tensors, got {device}")
    if stream is not None:
        return int(stream.cuda_stream)
    return torch._C._cuda_getCurrentRawStream(index)


def _status_word(dev_status, device, stream) -> torch.Tensor:
    """The caller's status word, or a new zeroed one, ordered on the call's
    stream (so the zeroing precedes the kernels that OR into it)."""
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, device)
        return dev_status
    with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(device)):
        return torch.zeros(1, dtype=torch.int32, device=device)


def _finish(rc: int, status: torch.Tensor, what: str, check: bool, check_device: bool, stream):
    if check and rc != 0:
        raise KdaError(rc, what)
    if check_device and rc == 0:
        (stream if stream is not None else torch.cuda.current_stream(status.device)).synchronize()
        bits = int(status.item())
        if bits != 0:
            raise KdaDeviceError(bits, what)
    return status


def kda_decode(output, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
               state_indices, gate_mode=GATE_SOFTPLUS, lower_bound=-5.0, dev_status=None,
               stream=None, check=True, check_device=False) -> torch.Tensor:
    """Advance the slot-indexed states over the packed tokens (see include/kda.h).

    Shapes (a leading batch axis of 1 is accepted): output [T, HV, V] fp32;
    q, k [T, H, K] bf16; v [T, HV, V] bf16; raw_gate [T, HV, K] fp32;
    beta_logits [T, HV] fp32; a_log [HV] fp32; dt_bias [HV, K] fp32;
    cu_seqlens [B+1] int32; state_pool [N, HV, K, V] fp32 (advanced in place);
    state_indices [B] int32.  Returns the device status word; raises KdaError
    on a negative C status when ``check`` (see the module docstring for
    ``dev_status`` and ``check_device``).
    """
    dev = state_pool.device
    T = q.shape[-3]
    H, K = q.shape[-2], q.shape[-1]
    HV, V = v.shape[-2], v.shape[-1]
    B = state_indices.shape[0]
    N = state_pool.shape[0]
    for t, n, dt in ((output, "output", torch.float32), (q, "q", torch.bfloat16),
                     (k, "k", torch.bfloat16), (v, "v", torch.bfloat16),
                     (raw_gate, "raw_gate", torch.float32),
                     (beta_logits, "beta_logits", torch.float32), (a_log, "a_log", torch.float32),
                     (dt_bias, "dt_bias", torch.float32), (cu_seqlens, "cu_seqlens", torch.int32),
                     (state_pool, "state_pool", torch.float32),
                     (state_indices, "state_indices", torch.int32)):
        _check(t, n, dt, dev)
    if tuple(state_pool.shape[1:]) != (HV, K, V):
        raise ValueError(f"state_pool shape {tuple(state_pool.shape)} != [N, {HV}, {K}, {V}]")
    if cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    status = _status_word(dev_status, dev, stream)
    rc = _lib.load().kda_decode(
        output.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), raw_gate.data_ptr(),
        beta_logits.data_ptr(), a_log.data_ptr(), dt_bias.data_ptr(), cu_seqlens.data_ptr(),
        state_pool.data_ptr(), state_indices.data_ptr(), int(gate_mode), float(lower_bound),
        B, T, H, HV, K, V, N, status.data_ptr(), _stream_handle(stream))
    return _finish(rc, status, "kda_decode", check, check_device, stream)


def kda_prefill(output, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
                state_indices, gate_mode=GATE_LOWER_BOUND, lower_bound=-5.0, dev_status=None,
                stream=None, check=True, check_device=False) -> torch.Tensor:
    """Whole-prompt prefill: the kda_decode recurrence computed 16 tokens at a
    time for the lower-bound gate with lower_bound >= -5; other gates run the
    token-by-token kernel.  Same tensors as kda_decode."""
    dev = state_pool.device
    T = q.shape[-3]
    H, K = q.shape[-2], q.shape[-1]
    HV, V = v.shape[-2], v.shape[-1]
    B = state_indices.shape[0]
    N = state_pool.shape[0]
    for t, n, dt in ((output, "output", torch.float32), (q, "q", torch.bfloat16),
                     (k, "k", torch.bfloat16), (v, "v", torch.bfloat16),
                     (raw_gate, "raw_gate", torch.float32),
                     (beta_logits, "beta_logits", torch.float32), (a_log, "a_log", torch.float32),
                     (dt_bias, "dt_bias", torch.float32), (cu_seqlens, "cu_seqlens", torch.int32),
                     (state_pool, "state_pool", torch.float32),
                     (state_indices, "state_indices", torch.int32)):
        _check(t, n, dt, dev)
    if tuple(state_pool.shape[1:]) != (HV, K, V):
        raise ValueError(f"state_pool shape {tuple(state_pool.shape)} != [N, {HV}, {K}, {V}]")
    if cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    status = _status_word(dev_status, dev, stream)
    rc = _lib.load().kda_prefill(
        output.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), raw_gate.data_ptr(),
        beta_logits.data_ptr(), a_log.data_ptr(), dt_bias.data_ptr(), cu_seqlens.data_ptr(),
        state_pool.data_ptr(), state_indices.data_ptr(), int(gate_mode), float(lower_bound),
        B, T, H, HV, K, V, N, status.data_ptr(), _stream_handle(stream))
    return _finish(rc, status, "kda_prefill", check, check_device, stream)


def kda_decode_ex(output, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
                  state_indices, gate_mode=GATE_SOFTPLUS, lower_bound=-5.0,
                  state_layout=STATE_K_FIRST, dev_status=None, stream=None, check=True,
                  check_device=False) -> torch.Tensor:
    """kda_decode with a chosen state layout (STATE_K_FIRST: tiles [K, V];
    STATE_V_FIRST: tiles [V, K]) and the output dtype taken from ``output``
    (float32 or bfloat16)."""
    dev = state_pool.device
    T = q.shape[-3]
    H, K = q.shape[-2], q.shape[-1]
    HV, V = v.shape[-2], v.shape[-1]
    B = state_indices.shape[0]
    N = state_pool.shape[0]
    if output.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"output: expected float32 or bfloat16, got {output.dtype}")
    out_dtype = OUTPUT_F32 if output.dtype == torch.float32 else OUTPUT_BF16
    _check(output, "output", output.dtype, dev)
    for t, n, dt in ((q, "q", torch.bfloat16), (k, "k", torch.bfloat16), (v, "v", torch.bfloat16),
                     (raw_gate, "raw_gate", torch.float32),
                     (beta_logits, "beta_logits", torch.float32), (a_log, "a_log", torch.float32),
                     (dt_bias, "dt_bias", torch.float32), (cu_seqlens, "cu_seqlens", torch.int32),
                     (state_pool, "state_pool", torch.float32),
                     (state_indices, "state_indices", torch.int32)):
        _check(t, n, dt, dev)
    tile = (K, V) if state_layout == STATE_K_FIRST else (V, K)
    if tuple(state_pool.shape[1:]) != (HV, *tile):
        raise ValueError(f"state_pool shape {tuple(state_pool.shape)} != [N, {HV}, {tile[0]}, {tile[1]}]")
    if cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    status = _status_word(dev_status, dev, stream)
    rc = _lib.load().kda_decode_ex(
        output.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), raw_gate.data_ptr(),
        beta_logits.data_ptr(), a_log.data_ptr(), dt_bias.data_ptr(), cu_seqlens.data_ptr(),
        state_pool.data_ptr(), state_indices.data_ptr(), int(gate_mode), float(lower_bound),
        int(state_layout), out_dtype, B, T, H, HV, K, V, N,
        status.data_ptr(), _stream_handle(stream))
    return _finish(rc, status, "kda_decode_ex", check, check_device, stream)


def block_workspace_size(B, n, Hd, nh, K, V, Kc) -> int:
    return int(_lib.load().kda_block_tkg_workspace_size(B, n, Hd, nh, K, V, Kc))


def kda_block_tkg(out, hidden, gamma_in, W_in, W_fb, W_gb, conv_w, A_log, dt_bias, gamma_o, W_o,
                  S, conv_state, scale, lower_bound, rms_norm_eps=1e-5, l2_eps=1e-6,
                  workspace=None, dev_status=None, stream=None, check=True,
                  check_device=False) -> torch.Tensor:
    """The fused KDA block (see include/kda.h).  ``workspace`` is a uint8 CUDA
    tensor of at least block_workspace_size(...) bytes; when None one is
    allocated here with torch (device memory plumbing only)."""
    dev = hidden.device
    B, n, Hd = hidden.shape
    _, nh, K, V = S.shape
    Kc = conv_state.shape[-1] + 1
    for t, name, dt in ((out, "out", torch.float32), (hidden, "hidden", torch.float32),
                        (gamma_in, "gamma_in", torch.float32), (W_in, "W_in", torch.bfloat16),
                        (W_fb, "W_fb", torch.bfloat16), (W_gb, "W_gb", torch.bfloat16),
                        (conv_w, "conv_w", torch.bfloat16), (A_log, "A_log", torch.float32),
                        (dt_bias, "dt_bias", torch.float32), (gamma_o, "gamma_o", torch.float32),
                        (W_o, "W_o", torch.bfloat16), (S, "S", torch.float32),
                        (conv_state, "conv_state", torch.float32)):
        _check(t, name, dt, dev)
    need = block_workspace_size(B, n, Hd, nh, K, V, Kc)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    status = _status_word(dev_status, dev, stream)
    rc = _lib.load().kda_block_tkg(
        out.data_ptr(), hidden.data_ptr(), gamma_in.data_ptr(), W_in.data_ptr(), W_fb.data_ptr(),
        W_gb.data_ptr(), conv_w.data_ptr(), A_log.data_ptr(), dt_bias.data_ptr(),
        gamma_o.data_ptr(), W_o.data_ptr(), S.data_ptr(), conv_state.data_ptr(), float(scale),
        float(lower_bound), float(rms_norm_eps), float(l2_eps), B, n, Hd, nh, K, V, Kc,
        workspace.data_ptr(), workspace.numel(), status.data_ptr(), _stream_handle(stream))
    return _finish(rc, status, "kda_block_tkg", check, check_device, stream)


def _check_rows(t: torch.Tensor, name: str, heads: int, D: int, device) -> int:
    """A [T, heads, D] bf16 tensor whose tokens may be strided (a view of a fused
    projection's output); returns the elements between two tokens."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != D:
        raise ValueError(f"{name} shape {tuple(shape)} != [T, {heads}, {D}]")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != D):
        raise ValueError(f"{name}: a token's rows must be contiguous (strides {s})")
    return s[0] if shape[0] > 1 else heads * D


def _check_cache(k_cache, v_cache, k_scale, v_scale, page_table, cu, what):
    """The tensors every call on a paged cache takes; returns (cache_dtype, B, HKV,
    D, page_size, num_pages, max_pages)."""
    dev, dtype, shape = k_cache.device, k_cache.dtype, k_cache.shape
    e4m3 = dtype is torch.float8_e4m3fn
    if not e4m3 and dtype is not torch.bfloat16:
        raise TypeError(f"k_cache: expected bfloat16 or float8_e4m3fn, got {dtype}")
    _check(k_cache, "k_cache", dtype, dev)
    _check(v_cache, "v_cache", dtype, dev)
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache {tuple(shape)} and v_cache {tuple(v_cache.shape)} must be "
                         "the same [num_pages, HKV, page_size, D]")
    N, HKV, page, D = shape
    if e4m3:
        if k_scale is None or v_scale is None:
            raise ValueError("an e4m3 cache needs k_scale and v_scale")
        rows = (N, HKV, page)
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _check(t, n, torch.float32, dev)
            if t.shape != rows:
                raise ValueError(f"{n} shape {tuple(t.shape)} != {rows}")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("a bf16 cache takes no scales")
    _check(page_table, "page_table", torch.int32, dev)
    _check(cu, what, torch.int32, dev)
    table = page_table.shape
    B = table[0]
    if len(table) != 2 or cu.numel() != B + 1:
        raise ValueError(f"page_table must be [B, max_pages] and {what} have B + 1 entries")
    return (CACHE_E4M3 if e4m3 else CACHE_BF16), B, HKV, D, page, N, table[1]


def _ptr(t):
    return None if t is None else t.data_ptr()


def kda_cache_append(k_cache, v_cache, k, v, cu_seqlens, seq_lens, page_table, k_scale=None,
                     v_scale=None, dev_status=None, stream=None, check=True,
                     check_device=False) -> torch.Tensor:
    """Write the new tokens' K and V rows into a paged cache (see include/kda.h).

    Shapes: k_cache, v_cache [num_pages, HKV, page_size, D] bf16 or
    float8_e4m3fn (then with k_scale, v_scale [num_pages, HKV, page_size] fp32);
    k, v [T, HKV, D] bf16, tokens may be strided; cu_seqlens [B+1] int32;
    seq_lens [B] int32 (the new tokens included); page_table [B, max_pages] int32.
    """
    dev = k_cache.device
    dtype, B, HKV, D, page, N, max_pages = _check_cache(k_cache, v_cache, k_scale, v_scale,
                                                        page_table, cu_seqlens, "cu_seqlens")
    ks, vs = _check_rows(k, "k", HKV, D, dev), _check_rows(v, "v", HKV, D, dev)
    if v.shape[0] != k.shape[0]:
        raise ValueError(f"k has {k.shape[0]} tokens, v {v.shape[0]}")
    _check(seq_lens, "seq_lens", torch.int32, dev)
    if seq_lens.numel() != B:
        raise ValueError("seq_lens must have B entries")
    status = _status_word(dev_status, dev, stream)
    rc = _lib.load().kda_cache_append(
        k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_scale), _ptr(v_scale), k.data_ptr(),
        v.data_ptr(), cu_seqlens.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(), dtype, B,
        k.shape[0], HKV, D, page, N, max_pages, ks, vs, status.data_ptr(), _stream_of(stream, dev))
    return _finish(rc, status, "kda_cache_append", check, check_device, stream)


def kda_cache_read(k_rows, v_rows, k_cache, v_cache, cu_rows, starts, page_table, k_scale=None,
                   v_scale=None, dev_status=None, stream=None, check=True,
                   check_device=False) -> torch.Tensor:
    """Rows of a paged cache back as dense bf16 rows: k_rows, v_rows [T, HKV, D]
    take request b's positions starts[b] .. (0 .. when ``starts`` is None)."""
    dev = k_cache.device
    dtype, B, HKV, D, page, N, max_pages = _check_cache(k_cache, v_cache, k_scale, v_scale,
                                                        page_table, cu_rows, "cu_rows")
    for t, n in ((k_rows, "k_rows"), (v_rows, "v_rows")):
        _check(t, n, torch.bfloat16, dev)
        if t.dim() != 3 or t.shape[1:] != (HKV, D) or t.shape != k_rows.shape:
            raise ValueError(f"{n} shape {tuple(t.shape)} != [T, {HKV}, {D}]")
    if starts is not None:
        _check(starts, "starts", torch.int32, dev)
        if starts.numel() != B:
            raise ValueError("starts must have B entries")
    status = _status_word(dev_status, dev, stream)
    rc = _lib.load().kda_cache_read(
        k_rows.data_ptr(), v_rows.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        _ptr(k_scale), _ptr(v_scale), cu_rows.data_ptr(), _ptr(starts), page_table.data_ptr(),
        dtype, B, k_rows.shape[0], HKV, D, page, N, max_pages, status.data_ptr(),
        _stream_of(stream, dev))
    return _finish(rc, status, "kda_cache_read", check, check_device, stream)


def paged_attention_workspace_size(B, T, max_tokens, H, HKV, D) -> int:
    return int(_lib.load().kda_paged_attention_workspace_size(B, T, max_tokens, H, HKV, D))


def kda_paged_attention(out, q, k_cache, v_cache, cu_seqlens, seq_lens, page_table, max_tokens,
                        scale=None, causal=True, window=0, k_scale=None, v_scale=None, lse=None,
                        workspace=None, dev_status=None, stream=None, check=True,
                        check_device=False) -> torch.Tensor:
    """Softmax attention of the new tokens over a paged cache that holds their own
    rows too (see include/kda.h).

    Shapes: out [T, H, D] bf16; q [T, H, D] bf16, tokens may be strided; the cache,
    cu_seqlens, seq_lens and page_table as kda_cache_append; lse [T, H] fp32 or None.
    ``max_tokens`` bounds every request's new tokens; ``scale`` defaults to
    D ** -0.5.  ``workspace`` is a uint8 CUDA tensor of at least
    paged_attention_workspace_size(...) bytes; when None one is allocated here.
    """
    dev = k_cache.device
    dtype, B, HKV, D, page, N, max_pages = _check_cache(k_cache, v_cache, k_scale, v_scale,
                                                        page_table, cu_seqlens, "cu_seqlens")
    shape = out.shape
    T, H = shape[0], shape[1]
    _check(out, "out", torch.bfloat16, dev)
    qs = _check_rows(q, "q", H, D, dev)
    if shape != q.shape:
        raise ValueError(f"out shape {tuple(shape)} != {tuple(q.shape)}")
    _check(seq_lens, "seq_lens", torch.int32, dev)
    if seq_lens.numel() != B:
        raise ValueError("seq_lens must have B entries")
    if lse is not None:
        _check(lse, "lse", torch.float32, dev)
        if lse.shape != (T, H):
            raise ValueError(f"lse shape {tuple(lse.shape)} != [{T}, {H}]")
    if workspace is None:
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(dev)):
            workspace = torch.empty(max(paged_attention_workspace_size(B, T, max_tokens, H, HKV, D), 1),
                                    dtype=torch.uint8, device=dev)
    else:
        _check(workspace, "workspace", torch.uint8, dev)
    status = _status_word(dev_status, dev, stream)
    rc = _lib.load().kda_paged_attention(
        out.data_ptr(), _ptr(lse), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        _ptr(k_scale), _ptr(v_scale), cu_seqlens.data_ptr(), seq_lens.data_ptr(),
        page_table.data_ptr(), float(D ** -0.5 if scale is None else scale), int(causal),
        int(window), dtype, B, T, int(max_tokens), H, HKV, D, page, N, max_pages, qs,
        workspace.data_ptr(), workspace.numel(), status.data_ptr(), _stream_of(stream, dev))
    return _finish(rc, status, "kda_paged_attention", check, check_device, stream)


def kda_verify_draft(tokens, accepted, target_probs, draft_probs, draft_tokens, accept_u, sample_u,
                     cu_drafts, dev_status=None, stream=None, check=True,
                     check_device=False) -> torch.Tensor:
    """Accept a prefix of each request's drafted tokens and draw the token after it
    (see include/kda.h).

    Shapes: tokens [N + B] int32, accepted [B] int32 (written); target_probs
    [N + B, V] fp32; draft_probs [N, V] fp32 or None (drafts proposed with
    certainty); draft_tokens [N] int32; accept_u [N], sample_u [B] fp32;
    cu_drafts [B+1] int32.  Rows of probabilities may be strided.
    """
    dev = target_probs.device
    B, N = accepted.shape[0], draft_tokens.shape[0]
    for t, n, dt, size in ((tokens, "tokens", torch.int32, N + B),
                           (accepted, "accepted", torch.int32, B),
                           (draft_tokens, "draft_tokens", torch.int32, N),
                           (accept_u, "accept_u", torch.float32, N),
                           (sample_u, "sample_u", torch.float32, B),
                           (cu_drafts, "cu_drafts", torch.int32, B + 1)):
        _check(t, n, dt, dev)
        if t.numel() != size:
            raise ValueError(f"{n}: expected {size} entries, got {t.numel()}")
    V = target_probs.shape[-1]
    strides = []
    for t, n, rows in ((target_probs, "target_probs", N + B), (draft_probs, "draft_probs", N)):
        if t is None:
            strides.append(V)
            continue
        if t.dtype != torch.float32:
            raise TypeError(f"{n}: expected {torch.float32}, got {t.dtype}")
        if t.device != dev:
            raise ValueError(f"{n}: expected device {dev}, got {t.device}")
        if t.shape != (rows, V) or (V > 1 and t.stride(1) != 1):
            raise ValueError(f"{n}: expected [{rows}, {V}] with contiguous rows, got {tuple(t.shape)}")
        strides.append(t.stride(0) if rows > 1 else V)
    status = _status_word(dev_status, dev, stream)
    rc = _lib.load().kda_verify_draft(
        tokens.data_ptr(), accepted.data_ptr(), target_probs.data_ptr(), _ptr(draft_probs),
        draft_tokens.data_ptr(), accept_u.data_ptr(), sample_u.data_ptr(), cu_drafts.data_ptr(),
        B, N, V, strides[0], strides[1], status.data_ptr(), _stream_of(stream, dev))
    return _finish(rc, status, "kda_verify_draft", check, check_device, stream)


def version() -> str:
    return _lib.load().kda_version().decode()
