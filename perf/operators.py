"""The cache, attention and draft-verification operators: cases, plain forms and 64-bit values.

Three operators that surround the KDA recurrence in one token-generation step:

  append / read   K and V rows into a paged cache (bf16, or e4m3 with one fp32 scale
                  per position and key head) and back into dense bf16 rows
  attention       a window or chunk of new tokens over that cache
  verify          drafted tokens against the target's probabilities, from given
                  uniform numbers

`own` selects the side: False computes the plain forms below with elementary torch
operations, True calls this repository's kernels.  A cache is [pages, key heads,
page size, head dim]; `table[b, i]` is the page of request b's positions
i * page .. i * page + page - 1 (-1: none); `lens[b]` counts the cached positions,
the new tokens' included.  Padding and ragged lengths follow from the case alone, the
values from the seed.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


def listed():
    return [
        # one decode step's new rows, one per request, quantised: latency
        dict(name="append_e4m3_64x1", op="append", B=64, n_lo=1, n_hi=1, ctx_lo=0, ctx_hi=2048, HKV=8, D=128, page=64, cache="e4m3", ragged=1),
        # the rows of several prompts at once, ragged, quantised: bandwidth
        dict(name="append_e4m3_prompts", op="append", B=9, n_lo=1000, n_hi=8191, ctx_lo=0, ctx_hi=0, HKV=8, D=128, page=64, cache="e4m3", ragged=2),
        # a short cached prefix read back to be handed on
        dict(name="read_e4m3_short", op="read", B=3, n_lo=17, n_hi=300, ctx_lo=0, ctx_hi=0, HKV=8, D=128, page=16, cache="e4m3", ragged=3),
        # long prefixes read back, ragged, from the middle of their sequences
        dict(name="read_e4m3_long", op="read", B=12, n_lo=500, n_hi=16000, ctx_lo=0, ctx_hi=900, HKV=8, D=128, page=64, cache="e4m3", ragged=4),
        # the smallest decode step: one request, one token, a short odd context
        dict(name="attn_decode_1x517", op="attention", B=1, n_lo=1, n_hi=1, ctx_lo=517, ctx_hi=517, H=32, HKV=8, D=128, page=64, cache="bf16", window=0, causal=True, ragged=5),
        # a batch of single tokens over quantised caches of ragged length
        dict(name="attn_decode_64_e4m3", op="attention", B=64, n_lo=1, n_hi=1, ctx_lo=1000, ctx_hi=8000, H=96, HKV=8, D=128, page=64, cache="e4m3", window=0, causal=True, ragged=6),
        # the largest decode step: long caches, one of them far longer than the rest could be
        dict(name="attn_decode_128_long", op="attention", B=128, n_lo=1, n_hi=1, ctx_lo=300, ctx_hi=20000, H=32, HKV=8, D=128, page=64, cache="bf16", window=0, causal=True, ragged=7),
        # drafted windows of 1 to 8 tokens, heads of 64, small pages
        dict(name="attn_window_32x8", op="attention", B=32, n_lo=1, n_hi=8, ctx_lo=200, ctx_hi=6000, H=32, HKV=4, D=64, page=16, cache="bf16", window=0, causal=True, ragged=8),
        # a chunk of a long prompt over what is cached already
        dict(name="attn_chunk_2048", op="attention", B=1, n_lo=2048, n_hi=2048, ctx_lo=28001, ctx_hi=28001, H=32, HKV=8, D=128, page=64, cache="bf16", window=0, causal=True, ragged=9),
        # whole prompts of ragged length, from a quantised cache
        dict(name="attn_prompts_e4m3", op="attention", B=4, n_lo=1500, n_hi=6001, ctx_lo=0, ctx_hi=0, H=32, HKV=8, D=128, page=128, cache="e4m3", window=0, causal=True, ragged=10),
        # a few short drafts, a small odd vocabulary: latency
        dict(name="verify_4x32001", op="verify", B=4, n_lo=0, n_hi=4, V=32001, drafts="probs", ragged=11),
        # a full batch of drafted windows over a large vocabulary
        dict(name="verify_256x131072", op="verify", B=256, n_lo=1, n_hi=7, V=131072, drafts="probs", ragged=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "attention", "verify"])
    seed = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    D = rng.choice([64, 128, 128])
    if op == "verify":
        V = _log(rng, 2000, 131072)
        B = _log(rng, 1, 256)
        n_hi = rng.randrange(0, 8)
        return dict(op=op, B=B, n_lo=rng.randrange(0, n_hi + 1), n_hi=n_hi, V=V, drafts=rng.choice(["probs", "probs", "point"]), ragged=seed)
    if op in ("append", "read"):
        B = _log(rng, 1, 64)
        n_hi = _log(rng, 1, 60000 // B)
        return dict(op=op, B=B, n_lo=max(1, n_hi // rng.choice([1, 2, 10])), n_hi=n_hi, ctx_lo=0, ctx_hi=rng.choice([0, _log(rng, 1, 4000)]), HKV=rng.choice([1, 2, 4, 8]), D=D, page=page, cache=cache, ragged=seed)
    HKV = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    kind = rng.choice(["token", "window", "chunk"])
    if kind == "token":
        B, n_hi = _log(rng, 1, 128), 1
    elif kind == "window":
        B, n_hi = _log(rng, 1, 64), rng.randrange(2, 9)
    else:
        B = _log(rng, 1, 6)
        n_hi = _log(rng, 9, min(4000, int((1.8e9 / (B * HKV * G)) ** 0.5)))
    # the plain form's score matrix stays below 1.8e9 values, the gathered cache below 1e9
    most = min(1.8e9 / (B * n_hi * HKV * G), 1e9 / (B * HKV * D), 30000) - n_hi
    ctx_hi = _log(rng, 1, max(2, int(most)))
    return dict(op=op, B=B, n_lo=rng.randrange(1, n_hi + 1), n_hi=n_hi, ctx_lo=rng.randrange(0, ctx_hi + 1), ctx_hi=ctx_hi, H=HKV * G, HKV=HKV, D=D, page=page, cache=cache,
                window=rng.choice([0, 0, _log(rng, 1, 4096)]), causal=rng.random() < 0.85, ragged=seed)


def _sizes(case):
    """(new tokens per request, tokens cached before them)."""
    r = random.Random(case["ragged"])
    n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])] if "ctx_lo" in case else None
    return n, ctx


def _cumulative(n):
    c = [0]
    for x in n:
        c.append(c[-1] + x)
    return c


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(case, lens, g):
    """A page table over a pool in random order, with pages that belong to nobody."""
    page = case["page"]
    need = [-(-x // page) for x in lens]
    width = max(max(need), 1) + 1
    pages = sum(need) + 3
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    at = torch.tensor(_cumulative(need)[:-1], device="cuda")[:, None] + torch.arange(width, device="cuda")[None]
    used = torch.arange(width, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(used, order[at.clamp_max(pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    return table.contiguous(), pages


def _cache(case, pages, g):
    shape = (pages, case["HKV"], case["page"], case["D"])
    if case["cache"] == "bf16":
        return torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16), None
    code = (torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16) * 130).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
    scale = torch.rand(shape[:3], device="cuda", generator=g) * 0.01 + 0.002
    return code, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, ctx = _sizes(case)
    B = case["B"]
    s = dict(case=case, B=B, n=n, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "verify":
        V, N = case["V"], sum(n)
        cu = _cumulative(n)
        s["cu"] = _ints(cu)
        s["target"] = torch.softmax(2.5 * torch.randn(N + B, V, device="cuda", generator=g), -1)
        # the draft model's distribution is near the target's at the same place
        rows = torch.tensor([cu[b] + b + i for b in range(B) for i in range(n[b])], dtype=torch.int64, device="cuda")
        near = torch.softmax(s["target"][rows].log_() + 0.7 * torch.randn(N, V, device="cuda", generator=g), -1)
        race = near / torch.empty_like(near).exponential_(1.0, generator=g)
        s["draft_tokens"] = race.argmax(-1).to(torch.int32) if N else torch.zeros(0, dtype=torch.int32, device="cuda")
        s["draft"] = near if case["drafts"] == "probs" else None
        s["accept_u"] = torch.rand(N, device="cuda", generator=g)
        s["sample_u"] = torch.rand(B, device="cuda", generator=g)
        s["tokens"] = torch.empty(N + B, dtype=torch.int32, device="cuda")
        s["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
        return s
    lens = [a + c for a, c in zip(n, ctx)]
    T = sum(n)
    HKV, D = case["HKV"], case["D"]
    s["lens_list"], s["T"] = lens, T
    s["cu"], s["lens"], s["start"] = _ints(_cumulative(n)), _ints(lens), _ints(ctx)
    s["table"], pages = _pages(case, lens, g)
    s["k_cache"], s["k_scale"] = _cache(case, pages, g)
    s["v_cache"], s["v_scale"] = _cache(case, pages, g)
    if case["op"] == "append":
        # rows of the fused projection that holds k and v side by side
        kv = torch.randn(T, 2, HKV, D, device="cuda", generator=g, dtype=torch.bfloat16)
        kv *= torch.exp(torch.randn(T, 2, HKV, 1, device="cuda", generator=g)).to(torch.bfloat16)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
    elif case["op"] == "read":
        s["k_out"] = torch.empty(T, HKV, D, device="cuda", dtype=torch.bfloat16)
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        s["q"] = torch.randn(T, case["H"], D, device="cuda", generator=g, dtype=torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(T, case["H"], device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _token_places(s):
    """Request and position of every packed new token."""
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    return b, s["lens"].long()[b] - n[b] + t - s["cu"].long()[b]


def _plain_append(s):
    page = s["case"]["page"]
    b, pos = _token_places(s)
    where = s["table"].long()[b, pos // page]
    off = pos % page
    if s["k_scale"] is None:
        s["k_cache"][where, :, off] = s["k"]
        s["v_cache"][where, :, off] = s["v"]
        return [s["k_cache"], s["v_cache"]]
    x = torch.stack([s["k"], s["v"]]).float()
    most = x.abs().amax(-1)
    scale = torch.where(most > 0, most / E4M3_MAX, torch.ones_like(most))
    code = (x / scale[..., None]).to(E4M3).view(torch.uint8)
    s["k_cache"].view(torch.uint8)[where, :, off] = code[0]
    s["v_cache"].view(torch.uint8)[where, :, off] = code[1]
    s["k_scale"][where, :, off] = scale[0]
    s["v_scale"][where, :, off] = scale[1]
    return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _rows(cache, scale, where, off):
    """fp32 rows [..., HKV, D] at (page, offset)."""
    if scale is None:
        return cache[where, :, off].float()
    return cache.view(torch.uint8)[where, :, off].view(E4M3).float() * scale[where, :, off][..., None]


def _plain_read(s):
    b, pos = _token_places(s)
    where, off = s["table"].long()[b, pos // s["case"]["page"]], pos % s["case"]["page"]
    return [_rows(s["k_cache"], s["k_scale"], where, off).bfloat16(), _rows(s["v_cache"], s["v_scale"], where, off).bfloat16()]


def _plain_attention(s):
    c = s["case"]
    B, H, HKV, D, page = s["B"], c["H"], c["HKV"], c["D"], c["page"]
    G, n_max, l_max = H // HKV, max(s["n"]), max(s["lens_list"])
    b, pos = _token_places(s)
    i = torch.arange(s["T"], device="cuda") - s["cu"].long()[b]
    at = torch.arange(l_max, device="cuda")
    there = at[None] < s["lens"][:, None]                                             # [B, L]
    where = s["table"].long()[:, at // page].clamp_min(0)
    off = (at % page)[None].expand(B, -1)
    k = _rows(s["k_cache"], s["k_scale"], where, off).permute(0, 2, 1, 3)              # [B, HKV, L, D]
    v = _rows(s["v_cache"], s["v_scale"], where, off).masked_fill_(~there[..., None, None], 0).permute(0, 2, 1, 3)
    q = torch.zeros(B, n_max, H, D, device="cuda")
    q[b, i] = s["q"].float() * D ** -0.5
    q = q.view(B, n_max, HKV, G, D).permute(0, 2, 1, 3, 4).reshape(B, HKV, n_max * G, D)
    x = torch.matmul(q, k.transpose(-1, -2))                                          # [B, HKV, n G, L]
    place = (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + torch.arange(n_max, device="cuda")[None]
    seen = there[:, None, :].expand(B, n_max, l_max)
    if c["causal"]:
        seen = seen & (at[None, None] <= place[..., None])
    if c["window"]:
        seen = seen & (at[None, None] > place[..., None] - c["window"])
    seen = seen[:, None, :, None, :].expand(B, 1, n_max, G, l_max)
    x.view(B, HKV, n_max, G, l_max).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min_(-1e30)
    total = x.sub_(top).exp_().sum(-1, keepdim=True)
    out = torch.matmul(x, v) / total.clamp_min(1e-30)
    lse = top + total.log()
    out = out.view(B, HKV, n_max, G, D).permute(0, 2, 1, 3, 4).reshape(B, n_max, H, D)[b, i]
    lse = lse.view(B, HKV, n_max, G).permute(0, 2, 1, 3).reshape(B, n_max, H)[b, i]
    return [out.bfloat16(), lse]


def _plain_verify(s):
    B, V = s["B"], s["case"]["V"]
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    N = s["draft_tokens"].numel()
    first = cu[:-1] + torch.arange(B, device="cuda")                                  # each request's first target row
    t = torch.arange(N, device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    x = s["draft_tokens"].long()
    p = s["target"][t + b, x].double()
    q = s["draft"][t, x].double() if s["draft"] is not None else torch.ones(N, device="cuda", dtype=torch.float64)
    yes = torch.zeros(B, max(max(s["n"]), 1), device="cuda", dtype=torch.int64)
    yes[b, t - cu[b]] = (s["accept_u"].double() * q < p).long()
    j = yes.cumprod(1).sum(1)
    w = s["target"][first + j].double()
    if N:
        rejected = (j < n)[:, None]
        d = (cu[:-1] + j).clamp_max(N - 1)
        if s["draft"] is not None:
            less = s["draft"][d].double()
        else:
            less = torch.zeros_like(w).scatter_(1, x[d][:, None], 1.0)
        w = torch.where(rejected, (w - less).clamp_min_(0), w)
    c = w.cumsum(1)
    token = (c > s["sample_u"].double()[:, None] * c[:, -1:]).int().argmax(1)
    tokens = torch.full((N + B,), -1, dtype=torch.int32, device="cuda")
    keep = (t - cu[b]) < j[b]
    tokens[t + b] = torch.where(keep, s["draft_tokens"], tokens[t + b])
    tokens[first + j] = token.int()
    return [tokens, j.int()]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention, "verify": _plain_verify}[op](s)
    import kda_decode_recurrence_gb300 as kda
    if op == "append":
        kda.kda_cache_append(s["k_cache"], s["v_cache"], s["k"], s["v"], s["cu"], s["lens"], s["table"], k_scale=s["k_scale"], v_scale=s["v_scale"], dev_status=s["status"])
        return [s["k_cache"], s["v_cache"]] + ([s["k_scale"], s["v_scale"]] if s["k_scale"] is not None else [])
    if op == "read":
        kda.kda_cache_read(s["k_out"], s["v_out"], s["k_cache"], s["v_cache"], s["cu"], s["start"], s["table"], k_scale=s["k_scale"], v_scale=s["v_scale"], dev_status=s["status"])
        return [s["k_out"], s["v_out"]]
    if op == "attention":
        c = s["case"]
        if "workspace" not in s:  # a server allocates it once for its largest step
            s["workspace"] = torch.empty(kda.paged_attention_workspace_size(s["B"], s["T"], max(s["n"]), c["H"], c["HKV"], c["D"]), dtype=torch.uint8, device="cuda")
        kda.kda_paged_attention(s["out"], s["q"], s["k_cache"], s["v_cache"], s["cu"], s["lens"], s["table"], max(s["n"]), causal=c["causal"], window=c["window"],
                                k_scale=s["k_scale"], v_scale=s["v_scale"], lse=s["lse"], workspace=s["workspace"], dev_status=s["status"])
        return [s["out"], s["lse"]]
    kda.kda_verify_draft(s["tokens"], s["accepted"], s["target"], s["draft"], s["draft_tokens"], s["accept_u"], s["sample_u"], s["cu"], dev_status=s["status"])
    return [s["tokens"], s["accepted"]]


# ---------------------------------------------------------------- work, exact values

def _visible(case):
    """(cache rows that some new token of their request attends, pairs of new token and key)."""
    n, ctx = _sizes(case)
    rows = pairs = 0
    for a, c in zip(n, ctx):
        L, W = a + c, case["window"]
        first = max(0, c - W + 1) if W else 0
        rows += L - first
        hi = [min(L, c + i + 1) if case["causal"] else L for i in range(a)]
        lo = [max(0, c + i - W + 1) if W else 0 for i in range(a)]
        pairs += sum(x - y for x, y in zip(hi, lo))
    return rows, pairs


def work(case):
    n, ctx = _sizes(case)
    if case["op"] == "verify":
        B, N = case["B"], sum(n)
        # each request's token is drawn from one target row and, unless all its drafts were taken, one draft row
        some = sum(1 for x in n if x)
        return {"bytes": 4 * case["V"] * (B + (some if case["drafts"] == "probs" else 0)) + 20 * N + 16 * B, "flops": 3 * case["V"] * B}
    T, HKV, D = sum(n), case["HKV"], case["D"]
    row = HKV * (2 * D if case["cache"] == "bf16" else D + 4)
    if case["op"] != "attention":
        return {"bytes": 2 * T * (HKV * D * 2 + row), "flops": 4 * T * HKV * D}
    rows, pairs = _visible(case)
    return {"bytes": 2 * rows * row + 2 * T * case["H"] * D * 2 + 4 * T * case["H"], "flops": 4 * D * case["H"] * pairs}


def _nearest_e4m3(y):
    """Nearest e4m3 value, ties to even, of y in 64 bits (|y| <= 448)."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))).clamp_(-6, 8) - 3)
    return torch.round(y / step) * step


def _dense64(s, b, name, lo, hi):
    """Rows lo..hi-1 of request b of the cache, [HKV, rows, D] in 64 bits."""
    page = s["case"]["page"]
    first, last = lo // page, -(-hi // page)
    ids = s["table"][b, first:last].long()
    x = s[name + "_cache"].view(torch.uint8)[ids].view(s[name + "_cache"].dtype).double() if s[name + "_scale"] is not None else s[name + "_cache"][ids].double()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][ids].double()[..., None]
    x = x.permute(1, 0, 2, 3).reshape(s["case"]["HKV"], -1, s["case"]["D"])
    return x[:, lo - first * page:hi - first * page]


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers
    if case["op"] == "attention" and _visible(case)[1] * case["H"] * case["D"] * 4 > 4e12:
        return None
    s = prepare(case, seed)
    n, ctx = _sizes(case)
    cu = _cumulative(n)
    HKV, D, page = case["HKV"], case["D"], case["page"]
    if case["op"] == "append":
        out = {}
        for name in ("k", "v"):
            x = s[name].double()
            if s["k_scale"] is None:
                code, scale = x, None
                held = s[name + "_cache"].double()
            else:
                most = x.abs().amax(-1)
                scale = torch.where(most > 0, most / 448.0, torch.ones_like(most))
                code = _nearest_e4m3(x / scale[..., None])
                held = s[name + "_cache"].double()
                held_scale = s[name + "_scale"].double()
            for b in range(case["B"]):
                pos = ctx[b] + torch.arange(n[b], device="cuda")
                ids = s["table"][b].long()[pos // page]
                held[ids, :, pos % page] = code[cu[b]:cu[b + 1]]
                if scale is not None:
                    held_scale[ids, :, pos % page] = scale[cu[b]:cu[b + 1]]
            out[name] = (held, held_scale if scale is not None else None)
        return [out["k"][0], out["v"][0]] + ([out["k"][1], out["v"][1]] if s["k_scale"] is not None else [])
    if case["op"] == "read":
        return [torch.cat([_dense64(s, b, name, ctx[b], ctx[b] + n[b]).transpose(0, 1) for b in range(case["B"])]) for name in ("k", "v")]
    H = case["H"]
    G, W = H // HKV, case["window"]
    out = torch.zeros(s["T"], H, D, device="cuda", dtype=torch.float64)
    lse = torch.full((s["T"], H), -math.inf, device="cuda", dtype=torch.float64)
    for b in range(case["B"]):
        L = n[b] + ctx[b]
        k, v = _dense64(s, b, "k", 0, L), _dense64(s, b, "v", 0, L)
        for i0 in range(0, n[b], 512):
            i1 = min(n[b], i0 + 512)
            p = ctx[b] + torch.arange(i0, i1, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")[None]
            hidden = (j > p) if case["causal"] else torch.zeros(1, 1, dtype=torch.bool, device="cuda")
            if W:
                hidden = hidden | (j <= p - W)
            for h in range(H):
                z = s["q"][cu[b] + i0:cu[b] + i1, h].double() @ k[h // G].T / math.sqrt(D)
                z = z.masked_fill(hidden, -math.inf)
                e = torch.logsumexp(z, -1)
                lse[cu[b] + i0:cu[b] + i1, h] = e
                out[cu[b] + i0:cu[b] + i1, h] = torch.exp(z - e[:, None].clamp_min(-1e300)) @ v[h // G]
    return [out, lse]
