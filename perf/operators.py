"""Operators that decide what a paged KV cache keeps, with their plain forms.

Four operators of a serving step over the paged cache ([num_blocks, Hkv, 16,
D], reached through block tables) that go beyond one query per sequence:

* ``tree``     attention of drafted tokens, arranged in a tree, over a cached
               prefix and over the drafts that each one may see;
* ``weights``  one decode step that also adds every cached token's attention
               weight to a running sum kept beside the cache;
* ``select``   which tokens of each head to keep under a budget: the first
               ones, the most recent ones, and the heaviest of the rest;
* ``compact``  the kept tokens (or the accepted path of a draft) moved
               together inside the cache, in place.

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through the framework's entry points.
"""
import math

import numpy as np
import torch

own = False
BS = 16


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one user, a short answer being drafted: latency of a verification step
        {"name": "tree 1 x 1000, 8 drafts", "op": "tree", "B": 1, "len": 1000, "ragged": False, "T": 8, "Tragged": False,
         "Hkv": 8, "G": 4, "D": 128, "fp8": False},
        # the ordinary serving batch: 64 sequences of U[1,2048] cached tokens, 16 drafts each
        {"name": "tree 64 x U[1,2048], 16 drafts", "op": "tree", "B": 64, "len": 2048, "ragged": True, "T": 16,
         "Tragged": False, "Hkv": 8, "G": 4, "D": 128, "fp8": False},
        # long contexts: 16 x 32K tokens, 32 drafts each
        {"name": "tree 16 x 32K, 32 drafts", "op": "tree", "B": 16, "len": 32701, "ragged": False, "T": 32, "Tragged": False,
         "Hkv": 8, "G": 4, "D": 128, "fp8": False},
        # an E4M3 cache under 64 / 8 heads, every sequence with its own length and draft size
        {"name": "tree fp8 32 x U[1,8192], U[1,64] drafts", "op": "tree", "B": 32, "len": 8192, "ragged": True, "T": 64,
         "Tragged": True, "Hkv": 8, "G": 8, "D": 128, "fp8": True},
        # one user, a decode step that keeps the weights
        {"name": "weights 1 x 700", "op": "weights", "B": 1, "len": 700, "ragged": False, "Hkv": 8, "G": 4, "D": 128,
         "fp8": False, "fresh": False},
        # the ordinary batch
        {"name": "weights 64 x U[1,2048]", "op": "weights", "B": 64, "len": 2048, "ragged": True, "Hkv": 8, "G": 4,
         "D": 128, "fp8": False, "fresh": False},
        # long contexts in an E4M3 cache, 64 / 8 heads
        {"name": "weights fp8 8 x 32K", "op": "weights", "B": 8, "len": 32768, "ragged": False, "Hkv": 8, "G": 8, "D": 128,
         "fp8": True, "fresh": False},
        # the ordinary batch cut to 512 tokens a head
        {"name": "select 64 x U[1,2048] to 512", "op": "select", "B": 64, "len": 2048, "ragged": True, "Hkv": 8,
         "budget": 512, "sink": 4, "recent": 128},
        # four long documents cut to a quarter
        {"name": "select 4 x 64K to 16K", "op": "select", "B": 4, "len": 65536, "ragged": False, "Hkv": 8, "budget": 16384,
         "sink": 4, "recent": 1024},
        # the accepted path of 16 drafts moved behind each of 64 prefixes
        {"name": "compact 64 drafts of 16", "op": "compact", "kind": "draft", "B": 64, "len": 2048, "ragged": True, "T": 16,
         "Hkv": 8, "D": 128, "fp8": False, "weights": False},
        # the ordinary batch after a selection of 512 tokens a head
        {"name": "compact 64 x U[1,2048] to 512", "op": "compact", "kind": "select", "B": 64, "len": 2048, "ragged": True,
         "budget": 512, "Hkv": 8, "D": 128, "fp8": False, "weights": True},
        # long contexts of an E4M3 cache halved
        {"name": "compact fp8 8 x 32K to 16K", "op": "compact", "kind": "select", "B": 8, "len": 32768, "ragged": False,
         "budget": 16384, "Hkv": 8, "D": 128, "fp8": True, "weights": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tree", "weights", "select", "compact"])
    Hkv, G, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    B = _log_int(rng, 1, 64)
    c = {"op": op, "B": B, "ragged": rng.random() < 0.7, "Hkv": Hkv}
    if op == "select":
        c["len"] = _log_int(rng, 1, min(65536, 4 * 8 * 65536 // (B * Hkv)))
        c["budget"] = _log_int(rng, 1, max(1, c["len"]))
        c["sink"] = rng.randint(0, c["budget"] // 8)
        c["recent"] = rng.randint(0, (c["budget"] - c["sink"]) // 2)
        return c
    c |= {"D": D, "fp8": rng.random() < 0.4}
    if op == "tree":
        T = _log_int(rng, 1, 64)
        c |= {"T": T, "Tragged": rng.random() < 0.5, "G": G}
        c["len"] = _log_int(rng, 1, min(32701, 16 * 32701 // B, 500_000_000 // (B * Hkv * G * T)))
    elif op == "weights":
        c |= {"G": G, "fresh": rng.random() < 0.3}
        c["len"] = _log_int(rng, 1, min(32768, 8 * 32768 // B))
    elif rng.random() < 0.5:
        c |= {"kind": "draft", "T": _log_int(rng, 1, 64), "weights": rng.random() < 0.3}
        c["len"] = _log_int(rng, 1, min(32768, 4 * 32768 // B))
    else:
        c |= {"kind": "select", "weights": rng.random() < 0.7}
        c["len"] = _log_int(rng, 1, min(32768, 4 * 32768 // B))
        c["budget"] = _log_int(rng, 1, max(1, c["len"]))
    return c


# ------------------------------------------------------------------ the inputs
def _spread(n, count, ragged):
    """`count` sizes: all n, or spread evenly over 1 .. n (which sequence has which is drawn)."""
    return 1 + (np.arange(count) * 2 + 1) * n // (2 * count) if ragged else np.full(count, n)


def _pool(case):
    """Blocks of the pool: a tenth more than the sequences and their drafts need."""
    return int(1.1 * np.sum(_spread(case["len"], case["B"], case["ragged"]) // BS + 1 + (case.get("T", 0) + BS - 1) // BS)) + 1


def _tables(lens, pool, g, dev):
    """Block tables over a scattered pool (entries past a sequence's last block are -1)."""
    nb = (lens + BS - 1) // BS
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(nb)[:-1]])).to(dev)
    j = torch.arange(int(nb.max()), device=dev)
    bt = perm[(off[:, None] + j).clamp(max=pool - 1)]
    return torch.where(j < torch.from_numpy(nb).to(dev)[:, None], bt, torch.full_like(bt, -1)).contiguous()


def _cache(case, pool, g, dev):
    shape = (pool, case["Hkv"], BS, case["D"])
    if not case["fp8"]:
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16), None
    scale = (5.5 / 448) * (1 + 0.125 * torch.arange(case["Hkv"], device=dev, dtype=torch.float32))
    x = torch.randn(shape, generator=g, device=dev)
    return x.div_(scale[:, None, None]).to(torch.float8_e4m3fn), scale


def _i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)


def _running_weights(shape, g, dev):
    """Sums of attention weights: a few tokens carry most of the weight, many were never attended (exact ties at zero)."""
    w = torch.rand(shape, generator=g, device=dev).pow_(6).mul_(3)
    return torch.where(w < 1e-3, torch.zeros_like(w), w)


def prepare(case, seed):
    dev = "cuda"
    rng = np.random.RandomState(seed % (1 << 32))
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}
    B, Hkv, op, pool = case["B"], case["Hkv"], case["op"], _pool(case)
    lens = rng.permutation(_spread(case["len"], B, case["ragged"]))
    if op == "tree":
        T = rng.permutation(_spread(case["T"], B, case["Tragged"]))
        cu = np.concatenate([[0], np.cumsum(T)])
        # node i of a tree hangs below one of the nodes before it (node 0 below the prefix's last token) and sees the
        # prefix, its ancestors and itself
        masks = np.zeros((B, case["T"]), np.uint64)
        masks[:, 0] = 1
        for i in range(1, case["T"]):
            up = rng.randint(max(0, i - 4), i, B)
            masks[:, i] = masks[np.arange(B), up] | np.uint64(1 << i)
        valid = np.arange(case["T"]) < T[:, None]
        s |= {"cu": _i32(cu, dev), "prefix": _i32(lens, dev), "max_q": int(T.max()),
              "mask": torch.from_numpy(masks[valid].view(np.int64)).to(dev)}
        s["q"] = torch.randn(int(cu[-1]), Hkv * case["G"], case["D"], generator=g, device=dev).mul_(1.5).bfloat16()
        s["tables"] = _tables(lens + T, pool, g, dev)
    else:
        s["lens"] = _i32(lens, dev)
        extra = case["T"] if case.get("kind") == "draft" else 0
        s["tables"] = _tables(lens + extra, pool, g, dev)
    if op == "weights":
        s["q"] = torch.randn(B, Hkv * case["G"], case["D"], generator=g, device=dev).mul_(1.5).bfloat16()
        s["seen"] = _i32(np.zeros(B) if case["fresh"] else lens - 1, dev)
    if op in ("tree", "weights"):
        s["out"] = torch.zeros_like(s["q"])
        s["scale"] = 1 / math.sqrt(case["D"])
    if op in ("weights", "select") or case.get("weights"):
        s["weights"] = _running_weights((pool, Hkv, BS), g, dev)
    if op != "select":
        s["k"], s["k_scale"] = _cache(case, pool, g, dev)
        s["v"], s["v_scale"] = _cache(case, pool, g, dev)
    if op == "select":
        s["keep"] = torch.zeros(B, Hkv, case["budget"], dtype=torch.int32, device=dev)
        s["keep_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
    if op == "compact" and case["kind"] == "draft":
        T = case["T"]
        n = rng.randint(1, min(T, 8) + 1, B)
        order = np.sort(np.argsort(rng.rand(B, T), axis=1)[:, :min(T, 8)], axis=1)  # an accepted path: ascending nodes
        s["start"] = s["lens"]
        s["keep"] = _i32(np.where(np.arange(order.shape[1]) < n[:, None], lens[:, None] + order, -1)[:, None, :], dev)
        s["keep_lens"] = _i32(n, dev)
    elif op == "compact":
        # what a selection leaves: the first 4, the last eighth and a random part of the rest, ascending
        n = np.minimum(lens, case["budget"])
        L = int(lens.max())
        pos = torch.arange(L, device=dev)
        score = torch.rand(B, Hkv, L, generator=g, device=dev)
        ln = s["lens"].long()[:, None, None]
        nn = torch.from_numpy(n).to(dev)[:, None, None]
        score = torch.where((pos < 4) | (pos >= ln - nn // 8), score + 2, score)
        score = torch.where(pos < ln, score, torch.full_like(score, -1.0))
        width = int(min(case["budget"], L))
        top = score.topk(width, dim=-1).indices
        top = torch.where(torch.arange(width, device=dev) < nn, top, torch.full_like(top, L)).sort(dim=-1).values
        keep = torch.full((B, Hkv, case["budget"]), -1, dtype=torch.int32, device=dev)
        keep[..., :width] = torch.where(top < L, top, torch.full_like(top, -1)).int()
        s["start"], s["keep"], s["keep_lens"] = None, keep, _i32(n, dev)
    return s


# ------------------------------------------------------------- the plain forms
def _values(cache, scale):
    """The cache's values in 32 bits."""
    if cache.dtype == torch.bfloat16:
        return cache.float()
    return cache.float() * scale[:, None, None]


def _rows(cache, scale, tables):
    """[B, Hkv, tokens, D] in 32 bits: every sequence's tokens through its block table."""
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    blocks = raw[tables.clamp(min=0).long()].view(cache.dtype)           # [B, nb, Hkv, 16, D]
    x = _values(blocks, scale).transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _softmax(score, allowed):
    """Softmax over the last axis of the allowed entries; rows that allow nothing are zero."""
    score = score.masked_fill_(~allowed, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = score.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = e.sum(-1, keepdim=True)
    return e.div_(torch.where(total == 0, torch.ones_like(total), total))


def _tree_plain(s):
    case = s["case"]
    B, Hkv, G, D = case["B"], case["Hkv"], case["G"], case["D"]
    T = s["max_q"]
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(T, device=cu.device)
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)             # [B, T]
    live = i < n[:, None]
    q = s["q"].float()[row].view(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    k, v = _rows(s["k"], s["k_scale"], s["tables"]), _rows(s["v"], s["v_scale"], s["tables"])
    pos = torch.arange(k.shape[2], device=cu.device)
    pre = s["prefix"].long()[:, None]
    node = (pos - pre)                                                   # [B, tokens]: the draft at a position
    bits = s["mask"][row]                                                # [B, T]
    sees = ((bits[:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1).bool()
    allowed = (pos < pre)[:, None, :] | (sees & ((node >= 0) & (node < n[:, None]))[:, None, :])
    score = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, G, T, -1)
    p = _softmax(score, allowed[:, None, None])
    o = (p.view(B, Hkv, G * T, -1) @ v).view(B, Hkv, G, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, Hkv * G, D)
    return o[live].bfloat16()


def _weights_plain(s):
    case = s["case"]
    B, Hkv, G, D = case["B"], case["Hkv"], case["G"], case["D"]
    k, v = _rows(s["k"], s["k_scale"], s["tables"]), _rows(s["v"], s["v_scale"], s["tables"])
    pos = torch.arange(k.shape[2], device=k.device)
    live = pos < s["lens"].long()[:, None]
    q = s["q"].float().view(B, Hkv, G, D)
    p = _softmax((q @ k.transpose(2, 3)).mul_(s["scale"]), live[:, None, None])
    out = (p @ v).view(B, Hkv * G, D).bfloat16()
    w = s["weights"]
    block = s["tables"].long()[:, pos // BS].clamp(min=0)                # [B, tokens]
    at = (block[:, None, :] * Hkv + torch.arange(Hkv, device=k.device)[:, None]) * BS + pos % BS
    old = torch.where(pos < s["seen"].long()[:, None], 1.0, 0.0)[:, None] * w.view(-1)[at]
    live = live[:, None].expand_as(at)
    w.view(-1)[at[live]] = (old + p.sum(2))[live]
    return {"out": out, "weights": w}


def _select_plain(s):
    case = s["case"]
    B, Hkv, n = case["B"], case["Hkv"], case["budget"]
    pos = torch.arange(s["tables"].shape[1] * BS, device=s["lens"].device)
    w = s["weights"][s["tables"].clamp(min=0).long()].transpose(1, 2).reshape(B, Hkv, -1)
    lens = s["lens"].long()[:, None]
    always = (pos < case["sink"]) | (pos >= lens - case["recent"])
    rank = torch.where(always[:, None], torch.full_like(w, math.inf), w)
    rank = torch.where((pos < lens)[:, None], rank, torch.full_like(w, -math.inf))
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :n]  # ties: the lowest position first
    got = torch.clamp(lens, max=n)                                        # [B, 1]
    width = order.shape[-1]
    last = torch.full_like(order, pos.numel())
    order = torch.where((torch.arange(width, device=w.device) < got)[:, None], order, last).sort(-1).values
    keep = torch.full((B, Hkv, n), -1, dtype=torch.int32, device=w.device)
    keep[..., :width] = torch.where(order < pos.numel(), order, torch.full_like(order, -1)).int()
    return {"keep": keep, "keep_lens": got[:, 0].int()}


def _compact_plain(s):
    case = s["case"]
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    keep = s["keep"].long().expand(B, Hkv, -1)
    i = torch.arange(keep.shape[-1], device=keep.device)
    live = (i < s["keep_lens"].long()[:, None])[:, None].expand_as(keep)
    to = i + (s["start"].long()[:, None] if s["start"] is not None else torch.zeros(B, 1, dtype=torch.long, device=i.device))
    head = torch.arange(Hkv, device=i.device)[None, :, None]
    row = torch.arange(B, device=i.device)[:, None, None]
    tables = s["tables"].long()

    def at(p):
        p = p.clamp(0, tables.shape[1] * BS - 1)
        return (tables[row, p // BS] * Hkv + head) * BS + p % BS

    src, dst = at(keep)[live], at(to[:, None].expand_as(keep))[live]
    got = {}
    for name in ("k", "v", "weights"):
        if name in s:
            x = s[name]
            flat = (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x).view(-1, D if name != "weights" else 1)
            flat[dst] = flat[src]
            got[name] = x
    return got


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"tree": _tree_plain, "weights": _weights_plain, "select": _select_plain, "compact": _compact_plain}[op](s)
    from paged_kv_cache_408_b200 import ops
    if op == "tree":
        if "ws" not in s:  # kept from step to step, as a serving loop keeps it
            s["ws"] = ops.alloc_tree_workspace(s["case"]["B"], s["q"].shape[1], s["max_q"], s["tables"].shape[1], s["k"])
        ops.decode_tree(s["out"], s["q"], s["cu"], s["prefix"], s["mask"], s["tables"], s["k"], s["v"], s["scale"],
                        s["max_q"], s["ws"], s["k_scale"], s["v_scale"])
        return s["out"]
    if op == "weights":
        if "ws" not in s:
            s["ws"] = ops.alloc_weights_workspace(s["case"]["B"], s["q"].shape[1], s["tables"].shape[1], s["k"])
        ops.decode_weights(s["out"], s["weights"], s["q"], s["k"], s["v"], s["tables"], s["lens"], s["scale"], s["ws"],
                           s["seen"], s["k_scale"], s["v_scale"])
        return {"out": s["out"], "weights": s["weights"]}
    if op == "select":
        ops.select_tokens(s["keep"], s["keep_lens"], s["weights"], s["tables"], s["lens"], s["case"]["sink"],
                          s["case"]["recent"])
        return {"keep": s["keep"], "keep_lens": s["keep_lens"]}
    ops.compact_kv(s["k"], s["v"], s["tables"], s["keep"], s["keep_lens"], s.get("weights"), s["start"])
    return {n: s[n] for n in ("k", "v", "weights") if n in s}


# ------------------------------------------------------------------- the floor
def work(case):
    """Each input read once, each output written once."""
    B, Hkv, op = case["B"], case["Hkv"], case["op"]
    lens = _spread(case["len"], B, case["ragged"])
    tokens = float(lens.sum())
    tables = tokens / BS * 4
    if op == "select":
        got = float(np.minimum(lens, case["budget"]).sum())
        return {"bytes": tokens * Hkv * 4 + tables + got * Hkv * 4 + B * 8, "flops": tokens * Hkv}
    eb = 1 if case["fp8"] else 2
    D = case["D"]
    if op == "tree":
        T = _spread(case["T"], B, case["Tragged"]).astype(float)
        Hq, drafts = Hkv * case["G"], float(T.sum())
        # a draft sees the prefix and about half of the drafts
        return {"bytes": (tokens + drafts) * Hkv * 2 * D * eb + tables + drafts * (Hq * D * 4 + 8),
                "flops": (tokens * drafts / B + float((T * T).sum()) / 2) * Hq * D * 4}
    if op == "weights":
        Hq = Hkv * case["G"]
        return {"bytes": tokens * Hkv * (2 * D * eb + 8) + tables + B * Hq * D * 4, "flops": tokens * Hq * D * 4}
    row = 2 * D * eb + (4 if case["weights"] else 0)
    if case["kind"] == "draft":
        n = min(case["T"], 8)
        kept = B * (n + 1) / 2
        moved = kept * (1 - n / case["T"] / 2) if case["T"] > 1 else 0.0  # nodes of the path that are not in place already
    else:
        n = np.minimum(lens, case["budget"])
        kept, moved = float(n.sum()), float(n[lens > n].sum())
    return {"bytes": moved * Hkv * row * 2 + kept * 4 * (Hkv if case["kind"] == "select" else 1) + tables + B * 8,
            "flops": moved * Hkv}


# -------------------------------------------------------------- the definition
def _tokens64(cache, scale, table, n):
    """[n, Hkv, D] in 64 bits: the first n tokens of one sequence."""
    p = torch.arange(n, device=table.device)
    b = table.long()[p // BS]
    x = cache[b, :, p % BS] if cache.dtype == torch.bfloat16 else cache.view(torch.uint8)[b, :, p % BS].view(cache.dtype)
    x = x.to(torch.float32).double()
    return x if scale is None else x * scale.double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "select":
        return None  # whole numbers
    if op == "compact":
        got = {n: s[n].to(torch.float32).double() for n in ("k", "v", "weights") if n in s}
        src = {n: x.clone() for n, x in got.items()}
        counts = s["keep_lens"].tolist()
        first = s["start"].tolist() if s["start"] is not None else [0] * case["B"]
        for b, n in enumerate(counts):
            for h in range(case["Hkv"]):
                a = s["keep"][b, h if s["keep"].shape[1] > 1 else 0, :n].long()
                z = torch.arange(first[b], first[b] + n, device=a.device)
                t = s["tables"][b].long()
                for name, x in got.items():
                    x[t[z // BS], h, z % BS] = src[name][t[a // BS], h, a % BS]
        return got
    Hkv, G, D = case["Hkv"], case["G"], case["D"]
    if op == "weights":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        w = s["weights"].double()
        for b, n in enumerate(s["lens"].tolist()):
            k, v = (_tokens64(s[c], s[c + "_scale"], s["tables"][b], n) for c in "kv")
            q = s["q"][b].double().view(Hkv, G, D)
            p = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * s["scale"], -1)
            out[b] = torch.einsum("hgt,thd->hgd", p, v).reshape(Hkv * G, D)
            t = torch.arange(n, device=w.device)
            blk = s["tables"][b].long()[t // BS]
            before = torch.where(t < int(s["seen"][b]), 1.0, 0.0).double()[:, None] * w[blk, :, t % BS]
            w[blk, :, t % BS] = before + p.sum(1).T
        return {"out": out, "weights": w}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    cu, pre = s["cu"].tolist(), s["prefix"].tolist()
    for b in range(case["B"]):
        T, P = cu[b + 1] - cu[b], pre[b]
        k, v = (_tokens64(s[c], s[c + "_scale"], s["tables"][b], P + T) for c in "kv")
        q = s["q"][cu[b]:cu[b + 1]].double().view(T, Hkv, G, D)
        bits = s["mask"][cu[b]:cu[b + 1]]
        see = torch.ones(T, P + T, dtype=torch.bool, device=q.device)
        see[:, P:] = ((bits[:, None] >> torch.arange(T, device=q.device)) & 1) == 1
        z = torch.einsum("ihgd,thd->hgit", q, k) * s["scale"]
        p = torch.softmax(z.masked_fill(~see, -math.inf), -1)
        out[cu[b]:cu[b + 1]] = torch.einsum("hgit,thd->ihgd", p, v).reshape(T, Hkv * G, D)
    return out
