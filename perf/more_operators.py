"""Latent attention and attention of drafted trees: cases, plain forms and 64-bit values.

Operators for a model's full-attention layers and its drafted tokens, next to the KDA
recurrence in a serving step:

  latent append    new tokens' latent rows (512 entries, normed on the way, and 64 of the
                   position) into a paged latent cache
  latent           attention of new tokens over that cache, every head reading the same
                   row (absorbed form): single tokens, windows, drafted trees
  expanded         attention over keys and values that were expanded from the latents,
                   per head 128 + 64 shared against 128, for prompts
  tree             attention of a tree of drafted tokens over a paged K/V cache

`own` selects the side: False computes the plain forms below with elementary torch
operations, True calls this repository's kernels.  `table[b, i]` is the page of request
b's positions i * page .. i * page + page - 1 (-1: none); `lens[b]` counts the cached
positions, the new tokens' included.  A tree is a mask of bits per new token: bit a of
token i says that i sees the request's new token a; all that was cached before is seen.
Padding, ragged lengths and trees follow from the case alone, the values from the seed.
"""
import math
import random

import torch

own = False

LATENT, ROPE = 512, 64            # entries of a latent row: what is attended, what tells the position
ROW = LATENT + ROPE
HEAD = 128                        # an expanded head's key entries (beside ROPE shared ones) and values
SCALE = (HEAD + ROPE) ** -0.5
E4M3 = torch.float8_e4m3fn
EPS = 1e-5


def listed():
    return [
        # one decode step's new latent rows, one per request: latency
        dict(name="latent_append_64x1", op="append", B=64, n_lo=1, n_hi=1, ctx_lo=0, ctx_hi=2048, page=64, norm=True, ragged=21),
        # the latent rows of several prompts at once, ragged: bandwidth
        dict(name="latent_append_prompts", op="append", B=9, n_lo=1000, n_hi=8191, ctx_lo=0, ctx_hi=0, page=64, norm=True, ragged=22),
        # the smallest decode step: one request, one token, 16 heads of a shard, a short odd context
        dict(name="latent_1x517", op="latent", B=1, n_lo=1, n_hi=1, ctx_lo=517, ctx_hi=517, H=16, page=64, tree=False, causal=True, ragged=23),
        # a batch of single tokens, all 96 heads
        dict(name="latent_decode_64_96h", op="latent", B=64, n_lo=1, n_hi=1, ctx_lo=1000, ctx_hi=8000, H=96, page=64, tree=False, causal=True, ragged=24),
        # the largest decode step: long caches of ragged length, 32 heads
        dict(name="latent_decode_128_long", op="latent", B=128, n_lo=1, n_hi=1, ctx_lo=300, ctx_hi=20000, H=32, page=64, tree=False, causal=True, ragged=25),
        # drafted windows of 1 to 8 tokens, small pages
        dict(name="latent_window_32x8", op="latent", B=32, n_lo=1, n_hi=8, ctx_lo=200, ctx_hi=6000, H=64, page=16, tree=False, causal=True, ragged=26),
        # drafted trees over latent caches
        dict(name="latent_tree_16x40", op="latent", B=16, n_lo=5, n_hi=40, ctx_lo=500, ctx_hi=6000, H=32, page=64, tree=True, causal=False, ragged=27),
        # a few prompts of odd lengths, a shard's heads
        dict(name="expanded_prompts_16h", op="expanded", B=5, n_lo=33, n_hi=1500, ctx_lo=0, ctx_hi=0, H=16, causal=True, ragged=28),
        # the largest: a chunk of a long prompt over what came before it, all heads
        dict(name="expanded_chunk_96h", op="expanded", B=1, n_lo=2048, n_hi=2048, ctx_lo=6001, ctx_hi=6001, H=96, causal=True, ragged=29),
        # one small tree over a short odd context: latency
        dict(name="tree_1x13", op="tree", B=1, n_lo=13, n_hi=13, ctx_lo=517, ctx_hi=517, H=32, HKV=8, D=128, page=64, cache="bf16", ragged=30),
        # a batch of trees
        dict(name="tree_32x60", op="tree", B=32, n_lo=8, n_hi=60, ctx_lo=1000, ctx_hi=8000, H=32, HKV=8, D=128, page=64, cache="bf16", ragged=31),
        # trees over a quantised cache, all heads
        dict(name="tree_16x32_e4m3", op="tree", B=16, n_lo=4, n_hi=32, ctx_lo=500, ctx_hi=12000, H=96, HKV=8, D=128, page=64, cache="e4m3", ragged=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "latent", "latent", "latent", "expanded", "expanded", "tree", "tree"])
    seed = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 64)
        n_hi = _log(rng, 1, 40000 // B)
        return dict(op=op, B=B, n_lo=max(1, n_hi // rng.choice([1, 2, 10])), n_hi=n_hi, ctx_lo=0, ctx_hi=rng.choice([0, _log(rng, 1, 4000)]), page=page,
                    norm=rng.random() < 0.7, ragged=seed)
    if op == "expanded":
        B, H = _log(rng, 1, 8), rng.choice([1, 4, 12, 16, 32, 64, 96])
        n_hi = _log(rng, 1, min(6000, int((4e8 / (B * H)) ** 0.5)))
        ctx_hi = rng.choice([0, _log(rng, 1, max(1, min(8000, int(1e9 / (B * H * n_hi)), 80000 // B)))])
        return dict(op=op, B=B, n_lo=rng.randrange(1, n_hi + 1), n_hi=n_hi, ctx_lo=rng.randrange(0, ctx_hi + 1), ctx_hi=ctx_hi, H=H, causal=rng.random() < 0.8, ragged=seed)
    kind = rng.choice(["token", "window", "tree"]) if op == "latent" else "tree"
    if kind == "token":
        B, n_hi = _log(rng, 1, 128), 1
    elif kind == "window":
        B, n_hi = _log(rng, 1, 48), rng.randrange(2, 9)
    else:
        B, n_hi = _log(rng, 1, 32), _log(rng, 2, 64)
    if op == "latent":
        H = rng.choice([1, 8, 12, 16, 32, 64, 96, 128])
        most = min(1.2e8 / (B * n_hi * H), 1.2e9 / (B * ROW), 24000) - n_hi
        ctx_hi = _log(rng, 1, max(2, int(most)))
        return dict(op=op, B=B, n_lo=rng.randrange(1, n_hi + 1), n_hi=n_hi, ctx_lo=rng.randrange(0, ctx_hi + 1), ctx_hi=ctx_hi, H=H, page=page,
                    tree=kind == "tree", causal=kind != "tree" and rng.random() < 0.85, ragged=seed)
    HKV, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128])
    G = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    most = min(6e8 / (B * n_hi * HKV * G), 1e9 / (B * HKV * D), 24000) - n_hi
    ctx_hi = _log(rng, 1, max(2, int(most)))
    return dict(op=op, B=B, n_lo=rng.randrange(1, n_hi + 1), n_hi=n_hi, ctx_lo=rng.randrange(0, ctx_hi + 1), ctx_hi=ctx_hi, H=HKV * G, HKV=HKV, D=D, page=page,
                cache=rng.choice(["bf16", "e4m3"]), ragged=seed)


def _sizes(case):
    """(new tokens per request, tokens cached before them)."""
    r = random.Random(case["ragged"])
    n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    return n, ctx


def _trees(case):
    """Per request and node the nodes it sees: itself and its ancestors (each node's parent is an
    earlier node or the cached text)."""
    r = random.Random(case["ragged"] + 1)
    trees = []
    for n in _sizes(case)[0]:
        seen = []
        for i in range(n):
            parent = r.randint(max(-1, i - 8), i - 1)
            seen.append((seen[parent] if parent >= 0 else set()) | {i})
        trees.append(seen)
    return trees


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
    code = (torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16) * 130).clamp_(-448, 448).to(E4M3)
    scale = torch.rand(shape[:3], device="cuda", generator=g) * 0.01 + 0.002
    return code, scale


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, ctx = _sizes(case)
    lens = [a + c for a, c in zip(n, ctx)]
    T, op = sum(n), case["op"]
    s = dict(case=case, B=case["B"], n=n, lens_list=lens, T=T, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    s["cu"], s["lens"] = _ints(_cumulative(n)), _ints(lens)
    if op == "expanded":
        Tk, H = sum(lens), case["H"]
        s["cu_k"] = _ints(_cumulative(lens))
        s["q"] = _normal(g, T, H, HEAD + ROPE)
        s["kv"] = _normal(g, Tk, H, 2 * HEAD)      # the expanding projection's output, key and value side by side
        s["k_pe"] = _normal(g, Tk, ROPE)
        s["out"] = torch.empty(T, H, HEAD, device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.empty(T, H, device="cuda")
        return s
    s["table"], pages = _pages(case, lens, g)
    if case.get("tree", op == "tree"):
        words = -(-max(n) // 32)
        bits = [[sum(1 << (a - 32 * w) for a in seen if a // 32 == w) for w in range(words)] for tree in _trees(case) for seen in tree]
        s["mask"] = torch.tensor(bits, dtype=torch.int64, device="cuda").to(torch.int32)
    if op == "tree":
        s["k_cache"], s["k_scale"] = _cache(case, pages, g)
        s["v_cache"], s["v_scale"] = _cache(case, pages, g)
        s["q"] = _normal(g, T, case["H"], case["D"])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(T, case["H"], device="cuda")
        return s
    s["cache"] = _normal(g, pages, case["page"], ROW)
    if op == "append":
        # columns of the fused projection that makes the latents beside the queries' part
        x = _normal(g, T, 448 + ROW) * torch.exp(torch.randn(T, 1, device="cuda", generator=g)).bfloat16()
        s["rows"] = x[:, 448:]
        s["gamma"] = 1 + 0.1 * torch.randn(LATENT, device="cuda", generator=g) if case["norm"] else None
        return s
    s["q"] = _normal(g, T, case["H"], ROW)
    s["out"] = torch.empty(T, case["H"], LATENT, device="cuda", dtype=torch.bfloat16)
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
    x = s["rows"]
    if s["gamma"] is not None:
        c = x[:, :LATENT].float()
        c = c * (c.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["gamma"]
        x = torch.cat([c.bfloat16(), x[:, LATENT:]], -1)
    s["cache"][s["table"].long()[b, pos // page], pos % page] = x
    return [s["cache"]]


def _seen(s, n_max, l_max):
    """[B, n_max, l_max]: which positions the new tokens see."""
    c, at = s["case"], torch.arange(l_max, device="cuda")
    n = s["cu"][1:] - s["cu"][:-1]
    ctx = s["lens"] - n
    there = (at[None] < s["lens"][:, None])[:, None, :].expand(s["B"], n_max, l_max)
    if "mask" in s:
        bits = torch.zeros(s["B"], n_max, s["mask"].shape[1], dtype=torch.int32, device="cuda")
        b, _ = _token_places(s)
        bits[b, torch.arange(s["T"], device="cuda") - s["cu"].long()[b]] = s["mask"]
        a = at[None] - ctx[:, None]                                                   # new token at a position
        word = (a.clamp(0, 32 * s["mask"].shape[1] - 1) // 32).long()
        bit = torch.gather(bits, 2, word[:, None, :].expand(s["B"], n_max, l_max)) >> (a % 32)[:, None, :]
        return there & ((a < 0)[:, None, :] | (bit & 1).bool())
    if c["causal"]:
        return there & (at[None, None] <= (ctx[:, None] + torch.arange(n_max, device="cuda")[None])[..., None])
    return there


def _softmax(x, seen, v):
    """Weights of the scores x [..., rows, L] where seen, times v; and their log-sum-exp."""
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min_(-1e30)
    total = x.sub_(top).exp_().sum(-1, keepdim=True)
    return torch.matmul(x, v) / total.clamp_min(1e-30), (top + total.log())[..., 0]


def _plain_latent(s):
    c = s["case"]
    B, H, page = s["B"], c["H"], c["page"]
    n_max, l_max = max(s["n"]), max(s["lens_list"])
    b, _ = _token_places(s)
    i = torch.arange(s["T"], device="cuda") - s["cu"].long()[b]
    at = torch.arange(l_max, device="cuda")
    rows = s["cache"][s["table"].long()[:, at // page].clamp_min(0), (at % page)[None].expand(B, -1)].float()   # [B, L, 576]
    rows.masked_fill_((at[None] >= s["lens"][:, None])[..., None], 0)
    q = torch.zeros(B, n_max, H, ROW, device="cuda")
    q[b, i] = s["q"].float() * SCALE
    x = torch.matmul(q.view(B, n_max * H, ROW), rows.transpose(-1, -2))
    seen = _seen(s, n_max, l_max)[:, :, None, :].expand(B, n_max, H, l_max).reshape(B, n_max * H, l_max)
    out, lse = _softmax(x, seen, rows[..., :LATENT])
    return [out.view(B, n_max, H, LATENT)[b, i].bfloat16(), lse.view(B, n_max, H)[b, i]]


def _plain_expanded(s):
    c = s["case"]
    H = c["H"]
    out = torch.empty(s["T"], H, HEAD, device="cuda")
    lse = torch.empty(s["T"], H, device="cuda")
    q0 = k0 = 0
    for n, L in zip(s["n"], s["lens_list"]):
        q = s["q"][q0:q0 + n].float().transpose(0, 1) * SCALE                             # [H, n, 192]
        kv = s["kv"][k0:k0 + L].float().transpose(0, 1)                                   # [H, L, 256]
        k = torch.cat([kv[..., :HEAD], s["k_pe"][k0:k0 + L].float()[None].expand(H, -1, -1)], -1)
        seen = torch.ones(1, 1, dtype=torch.bool, device="cuda")
        if c["causal"]:
            seen = torch.arange(L, device="cuda")[None] <= (L - n + torch.arange(n, device="cuda"))[:, None]
        o, e = _softmax(torch.matmul(q, k.transpose(-1, -2)), seen, kv[..., HEAD:])
        out[q0:q0 + n], lse[q0:q0 + n] = o.transpose(0, 1), e.transpose(0, 1)
        q0, k0 = q0 + n, k0 + L
    return [out.bfloat16(), lse]


def _rows(cache, scale, where, off):
    """fp32 rows [..., HKV, D] at (page, offset)."""
    if scale is None:
        return cache[where, :, off].float()
    return cache.view(torch.uint8)[where, :, off].view(E4M3).float() * scale[where, :, off][..., None]


def _plain_tree(s):
    c = s["case"]
    B, H, HKV, D, page = s["B"], c["H"], c["HKV"], c["D"], c["page"]
    G, n_max, l_max = H // HKV, max(s["n"]), max(s["lens_list"])
    b, _ = _token_places(s)
    i = torch.arange(s["T"], device="cuda") - s["cu"].long()[b]
    at = torch.arange(l_max, device="cuda")
    where = s["table"].long()[:, at // page].clamp_min(0)
    off = (at % page)[None].expand(B, -1)
    beyond = (at[None] >= s["lens"][:, None])[..., None, None]
    k = _rows(s["k_cache"], s["k_scale"], where, off).permute(0, 2, 1, 3)                 # [B, HKV, L, D]
    v = _rows(s["v_cache"], s["v_scale"], where, off).masked_fill_(beyond, 0).permute(0, 2, 1, 3)
    q = torch.zeros(B, n_max, H, D, device="cuda")
    q[b, i] = s["q"].float() * D ** -0.5
    q = q.view(B, n_max, HKV, G, D).permute(0, 2, 1, 3, 4).reshape(B, HKV, n_max * G, D)
    x = torch.matmul(q, k.transpose(-1, -2))
    seen = _seen(s, n_max, l_max)[:, None, :, None, :].expand(B, HKV, n_max, G, l_max).reshape(B, HKV, n_max * G, l_max)
    out, lse = _softmax(x, seen, v)
    out = out.view(B, HKV, n_max, G, D).permute(0, 2, 1, 3, 4).reshape(B, n_max, H, D)[b, i]
    lse = lse.view(B, HKV, n_max, G).permute(0, 2, 1, 3).reshape(B, n_max, H)[b, i]
    return [out.bfloat16(), lse]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _plain_append, "latent": _plain_latent, "expanded": _plain_expanded, "tree": _plain_tree}[op](s)
    import kda_decode_recurrence_gb300 as kda
    c = s["case"]
    if op == "append":
        kda.kda_latent_append(s["cache"], s["rows"], s["cu"], s["lens"], s["table"], gamma=s["gamma"], eps=EPS, dev_status=s["status"])
        return [s["cache"]]
    if "workspace" not in s:  # a server allocates it once for its largest step
        size = {"latent": lambda: kda.latent_attention_workspace_size(s["B"], s["T"], c["H"]),
                "expanded": lambda: kda.latent_expanded_workspace_size(s["B"], s["T"], c["H"]),
                "tree": lambda: kda.tree_attention_workspace_size(s["B"], s["T"], max(s["n"]), c["H"], c["HKV"], c["D"])}[op]()
        s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    if op == "latent":
        kda.kda_latent_attention(s["out"], s["q"], s["cache"], s["cu"], s["lens"], s["table"], causal=c["causal"], tree_mask=s.get("mask"), lse=s["lse"],
                                 workspace=s["workspace"], dev_status=s["status"])
    elif op == "expanded":
        kda.kda_latent_expanded(s["out"], s["q"], s["kv"], s["k_pe"], s["cu"], s["cu_k"], causal=c["causal"], lse=s["lse"], workspace=s["workspace"],
                                dev_status=s["status"])
    else:
        kda.kda_tree_attention(s["out"], s["q"], s["k_cache"], s["v_cache"], s["cu"], s["lens"], s["table"], s["mask"], max(s["n"]), k_scale=s["k_scale"],
                               v_scale=s["v_scale"], lse=s["lse"], workspace=s["workspace"], dev_status=s["status"])
    return [s["out"], s["lse"]]


# ---------------------------------------------------------------- work, exact values

def _pairs(case):
    """Pairs of a new token and a position that it sees."""
    n, ctx = _sizes(case)
    if case.get("tree", case["op"] == "tree"):
        return sum(c * len(tree) + sum(len(seen) for seen in tree) for c, tree in zip(ctx, _trees(case)))
    return sum(a * c + (a * (a + 1) // 2 if case["causal"] else a * a) for a, c in zip(n, ctx))


def work(case):
    n, ctx = _sizes(case)
    T, Tk, op = sum(n), sum(n) + sum(ctx), case["op"]
    if op == "append":
        return {"bytes": 2 * T * ROW * 2 + (4 * LATENT if case["norm"] else 0), "flops": 4 * T * LATENT if case["norm"] else 0}
    H, pairs = case["H"], _pairs(case)
    mask = T * 4 * -(-max(n) // 32) if case.get("tree", op == "tree") else 0
    if op == "latent":
        return {"bytes": Tk * ROW * 2 + T * H * (ROW + LATENT) * 2 + 4 * T * H + mask, "flops": 2 * (ROW + LATENT) * H * pairs}
    if op == "expanded":
        return {"bytes": Tk * (H * 2 * HEAD + ROPE) * 2 + T * H * (2 * HEAD + ROPE) * 2 + 4 * T * H, "flops": 2 * (2 * HEAD + ROPE) * H * pairs}
    HKV, D = case["HKV"], case["D"]
    row = HKV * (2 * D if case["cache"] == "bf16" else D + 4)
    return {"bytes": 2 * Tk * row + 2 * T * H * D * 2 + 4 * T * H + mask, "flops": 4 * D * H * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    n, ctx = _sizes(case)
    cu, op = _cumulative(n), case["op"]
    if op == "append":
        held, x = s["cache"].double(), s["rows"].double()
        if s["gamma"] is not None:
            rms = torch.sqrt((x[:, :LATENT] ** 2).sum(-1) / LATENT + EPS)
            x[:, :LATENT] = x[:, :LATENT] / rms[:, None] * s["gamma"].double()
        for b in range(case["B"]):
            p = ctx[b] + torch.arange(n[b], device="cuda")
            held[s["table"][b].long()[p // case["page"]], p % case["page"]] = x[cu[b]:cu[b + 1]]
        return [held]
    H = case["H"]
    if _pairs(case) * H * ROW * 4 > 4e12:
        return None
    trees = _trees(case) if "mask" in s else None
    cu_k = _cumulative([a + c for a, c in zip(n, ctx)])
    out = torch.zeros(*s["out"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full((s["T"], H), -math.inf, device="cuda", dtype=torch.float64)
    for b in range(case["B"]):
        L = n[b] + ctx[b]
        hidden = torch.zeros(n[b], L, dtype=torch.bool, device="cuda")
        if trees is not None:
            look = torch.ones(n[b], n[b], dtype=torch.bool)
            for i, nodes in enumerate(trees[b]):
                look[i, list(nodes)] = False
            hidden[:, ctx[b]:] = look.cuda()
        elif case["causal"]:
            hidden = torch.arange(L, device="cuda")[None] > ctx[b] + torch.arange(n[b], device="cuda")[:, None]

        def dense(x):
            ids = s["table"][b, :-(-L // case["page"])].long()
            return (x.view(torch.uint8)[ids].view(x.dtype) if x.dtype == E4M3 else x[ids]).double()

        if op == "latent":
            rows = dense(s["cache"]).reshape(-1, ROW)[:L]
        elif op == "tree":
            k, v = dense(s["k_cache"]), dense(s["v_cache"])
            if s["k_scale"] is not None:
                k, v = k * dense(s["k_scale"])[..., None], v * dense(s["v_scale"])[..., None]
            k, v = (x.permute(1, 0, 2, 3).reshape(case["HKV"], -1, case["D"])[:, :L] for x in (k, v))
        for h in range(H):
            if op == "latent":
                key, value, scale = rows, rows[:, :LATENT], 1 / math.sqrt(HEAD + ROPE)
            elif op == "expanded":
                part = slice(cu_k[b], cu_k[b + 1])
                key = torch.cat([s["kv"][part, h, :HEAD], s["k_pe"][part]], 1).double()
                value, scale = s["kv"][part, h, HEAD:].double(), 1 / math.sqrt(HEAD + ROPE)
            else:
                g = h // (H // case["HKV"])
                key, value, scale = k[g], v[g], 1 / math.sqrt(case["D"])
            z = (s["q"][cu[b]:cu[b + 1], h].double() @ key.T * scale).masked_fill(hidden, -math.inf)
            e = torch.logsumexp(z, -1)
            lse[cu[b]:cu[b + 1], h] = e
            out[cu[b]:cu[b + 1], h] = torch.exp(z - e[:, None].clamp_min(-1e300)) @ value
    return [out, lse]
