"""Cases of speculative and streaming decoding over the paged KV cache.

Five operators, used one after another by a program that serves a model with
draft tokens over a paged cache of heads of 512 dimensions:

  resize    gives each sequence the pages its next tokens need and takes back
            the pages behind a sequence that got shorter
  append    writes the new tokens' keys and values into the pages, as bf16 or
            rounded to E4M3 with per-tensor scales
  tree      attention of the drafted tokens (a tree, or a plain run of tokens)
            over the cache, with an optional window and first positions that
            stay visible, bf16 or E4M3 cache
  compact   moves the accepted tokens' rows together after the verification
  fork      makes every sequence a child of some sequence: whole pages are
            shared by count, a page that is still filling is copied, pages
            nobody refers to any more are free again

Each has a plain form here in elementary torch operations.
"""
import math
import random

import numpy as np
import torch

own = False

D = 512
DEV = "cuda"
NEG = float("-inf")


# ------------------------------------------------------------------- the cases

def listed():
    """Sizes: 8 query heads over 4 KV heads, pages of 64, caches of 4,096, 16,384
    and 28,672 positions and batches of 1, 16 and 64 are the decode workloads of
    this repository; 32 over 4 are its prefill head counts."""
    return [
        # one user, a small tree of drafts: the step's latency counts
        {"name": "tree_b1_kv4096_t8", "op": "tree", "batch": 1, "nodes": 8, "hq": 8, "hk": 4, "kv": 4096,
         "page": 64, "window": 0, "sinks": 0, "tree": True, "fp8": False, "ragged": False},
        # a batch of users with large trees and contexts of different lengths: the cache is read once for 128 rows a KV head
        {"name": "tree_b16_kv28672_t64", "op": "tree", "batch": 16, "nodes": 64, "hq": 8, "hk": 4, "kv": 28672,
         "page": 64, "window": 0, "sinks": 0, "tree": True, "fp8": False, "ragged": True},
        # many users, an 8-bit cache, middle-sized trees
        {"name": "tree_fp8_b64_kv16384_t16", "op": "tree", "batch": 64, "nodes": 16, "hq": 8, "hk": 4, "kv": 16384,
         "page": 64, "window": 0, "sinks": 0, "tree": True, "fp8": True, "ragged": False},
        # a streaming session's next piece of text: a window plus the first tokens, 8 query heads a KV head, an odd number of tokens
        {"name": "sinks_b8_kv16384_q75_w4096", "op": "tree", "batch": 8, "nodes": 75, "hq": 32, "hk": 4, "kv": 16384,
         "page": 64, "window": 4096, "sinks": 4, "tree": False, "fp8": False, "ragged": True},
        # one decode step's token of each sequence
        {"name": "append_b16_t1", "op": "append", "batch": 16, "tokens": 1, "hq": 8, "hk": 4, "kv": 4096, "page": 64,
         "fp8": False, "ragged": False},
        # prompt pieces of a batch go into an 8-bit cache
        {"name": "append_fp8_b8_t4096", "op": "append", "batch": 8, "tokens": 4096, "hq": 32, "hk": 4, "kv": 16384,
         "page": 64, "fp8": True, "ragged": True},
        # one layer's cache after a verification step
        {"name": "compact_b16_t16", "op": "compact", "batch": 16, "tokens": 16, "accept": 6, "layers": 1, "hk": 4,
         "kv": 4096, "page": 64, "fp8": False, "ragged": False},
        # all layers at once, larger trees
        {"name": "compact_b64_t64_l8", "op": "compact", "batch": 64, "tokens": 64, "accept": 17, "layers": 8, "hk": 4,
         "kv": 1024, "page": 64, "fp8": False, "ragged": True},
        # a beam of four
        {"name": "fork_b4_kv4096", "op": "fork", "batch": 4, "children": 4, "parents": 2, "layers": 1, "hk": 4,
         "kv": 4096, "page": 64, "fp8": False},
        # sixteen prompts, each sampled several times, all layers
        {"name": "fork_b16_c64_kv4096_l8", "op": "fork", "batch": 16, "children": 64, "parents": 16, "layers": 8,
         "hk": 4, "kv": 4096, "page": 64, "fp8": False},
        # every decode step asks for room for its drafts
        {"name": "resize_b16_kv4096", "op": "resize", "batch": 16, "kv": 4096, "page": 64, "grow": 9, "spare": 256},
        # a large server's whole pool: hundreds of sequences grow, shrink and end
        {"name": "resize_b512_kv28672", "op": "resize", "batch": 512, "kv": 28672, "page": 64, "grow": 8192,
         "spare": 65536},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "append", "compact", "fork", "resize"])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    hq, hk = rng.choice([(8, 4), (8, 4), (32, 4), (16, 1), (12, 4), (4, 4), (8, 1)])
    if op == "tree":
        c = {"op": op, "batch": _log(rng, 1, 64), "nodes": _log(rng, 1, 128), "hq": hq, "hk": hk,
             "kv": _log(rng, 130, 28672), "page": page, "window": 0, "sinks": 0, "tree": rng.random() < 0.6,
             "fp8": rng.random() < 0.4, "ragged": rng.random() < 0.5}
        if rng.random() < 0.4:
            c["window"] = _log(rng, 1, 8192)
            c["sinks"] = rng.choice([0, 1, 4, rng.randint(1, 300)])
        most = work(listed()[1])
        while c["batch"] > 1 and (work(c)["bytes"] > most["bytes"] or work(c)["flops"] > most["flops"]):
            c["batch"] = (c["batch"] + 1) // 2
        return c
    if op == "append":
        c = {"op": op, "batch": _log(rng, 1, 64), "tokens": _log(rng, 1, 4096), "hq": hq, "hk": hk, "kv": 0,
             "page": page, "fp8": rng.random() < 0.5, "ragged": rng.random() < 0.5}
        while c["batch"] * c["tokens"] * hk > 8 * 4096 * 4 or c["batch"] * c["tokens"] * (hq + 2 * hk) > 8 * 4096 * 40:
            c["batch"], c["tokens"] = (c["batch"] + 1) // 2, (c["tokens"] + 1) // 2
        c["kv"] = c["tokens"] + _log(rng, 1, 4096)
        return c
    if op == "compact":
        t = _log(rng, 1, 128)
        c = {"op": op, "batch": _log(rng, 1, 64), "tokens": t, "accept": rng.randint(1, min(t, 24)),
             "layers": rng.choice([1, 2, 4, 8]), "hk": hk, "kv": t + _log(rng, 1, 1024), "page": page,
             "fp8": rng.random() < 0.5, "ragged": rng.random() < 0.5}
        while c["batch"] * c["accept"] * c["layers"] * hk > 64 * 17 * 8 * 4:
            c["batch"] = (c["batch"] + 1) // 2
        return c
    if op == "fork":
        b = _log(rng, 1, 16)
        return {"op": op, "batch": b, "children": _log(rng, 1, 64), "parents": rng.randint(1, b),
                "layers": rng.choice([1, 2, 4, 8]), "hk": rng.choice([1, 4]), "kv": _log(rng, 1, 4096),
                "page": rng.choice([16, 32, 64]), "fp8": rng.random() < 0.5}
    kv = _log(rng, 64, 28672)
    return {"op": op, "batch": _log(rng, 1, 512), "kv": kv, "page": page, "grow": rng.randint(1, kv),
            "spare": _log(rng, 8, 65536)}


# ------------------------------------------------- lengths and work of one case

def _lens(c, least=1):
    """The lengths of the sequences, from the case alone."""
    kv, b = c["kv"], c["batch"]
    if not c.get("ragged"):
        return [kv] * b
    return [max(least, kv - (i * 7919 + 13) % max(1, kv // 2)) for i in range(b)]


def _counts(c, most):
    """How many of `most` new tokens each sequence has."""
    if not c.get("ragged"):
        return [most] * c["batch"]
    return [max(1, most - (i * 31) % max(1, (most + 1) // 2)) for i in range(c["batch"])]


def _fork_plan(c):
    """(lengths of the sequences, parent of each child), from the case alone."""
    r = random.Random(c["kv"] * 1000003 + c["children"] * 1009 + c["batch"])
    lens = [max(1, c["kv"] - r.randint(0, max(0, c["kv"] // 4))) for _ in range(c["batch"])]
    return lens, [r.randrange(c["parents"]) for _ in range(c["children"])]


def _resize_plan(c):
    """(lengths now, lengths then): half grow, some shrink, a few end."""
    r = random.Random(c["kv"] * 1000003 + c["grow"] * 1009 + c["batch"])
    old = [r.randint(1, c["kv"]) for _ in range(c["batch"])]
    new, room = [], c["spare"]
    for n in old:
        k, pages = r.random(), lambda x: -(-x // c["page"])
        m = n + r.randint(1, c["grow"]) if k < 0.6 else r.randint(0, n) if k < 0.8 else 0 if k < 0.85 else n
        if m > n:
            if pages(m) - pages(n) > room:
                m = n
            else:
                room -= pages(m) - pages(n)
        new.append(m)
    return old, new


def work(case):
    c, page = case, case["page"]
    if c["op"] == "tree":
        lens, cnt = _lens(c, c["nodes"]), _counts(c, c["nodes"])
        elt, g = (1 if c["fp8"] else 2), c["hq"] // c["hk"]
        b = f = 0
        for n, t in zip(lens, cnt):
            seen = n if not c["window"] else min(n, c["window"] + t + c["sinks"])
            pairs = t * (n if not c["window"] else min(n, c["window"] + c["sinks"]))
            b += seen * c["hk"] * D * elt * 2 + t * c["hq"] * D * 4
            f += pairs * c["hk"] * g * D * 4
        return {"bytes": b, "flops": f}
    if c["op"] == "append":
        n = sum(_counts(c, c["tokens"])) * c["hk"] * D * 2
        return {"bytes": n * (2 + (1 if c["fp8"] else 2)), "flops": 0}
    if c["op"] == "compact":
        moved = sum(min(c["accept"], t) for t in _counts(c, c["tokens"]))
        return {"bytes": moved * c["layers"] * c["hk"] * D * (1 if c["fp8"] else 2) * 2 * 2, "flops": 0}
    if c["op"] == "fork":
        lens, parents = _fork_plan(c)
        row = c["hk"] * D * (1 if c["fp8"] else 2) * 2 * c["layers"]
        rows = sum(lens[p] % page for i, p in enumerate(parents) if p in parents[:i])
        pages = sum(-(-n // page) for n in lens) + sum(-(-lens[p] // page) for p in parents)
        return {"bytes": 2 * rows * row + 4 * pages + 8 * _pool(c), "flops": 0}
    old, new = _resize_plan(c)
    pages = sum(-(-n // page) for n in old) + sum(-(-n // page) for n in new)
    return {"bytes": 4 * pages + 8 * _pool(c), "flops": 0}


# ------------------------------------------------------------------- the inputs

def _pool(c):
    """Pages of the pool."""
    page = c["page"]
    if c["op"] == "fork":
        lens, parents = _fork_plan(c)
        return sum(-(-n // page) for n in lens) + len(parents) + 16
    if c["op"] == "resize":
        return sum(-(-n // page) for n in _resize_plan(c)[0]) + c["spare"]
    return c["batch"] * -(-c["kv"] // page) + 8


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _cache(shape, fp8, g):
    """Cached rows as a model leaves them: roughly normal values, bf16 or E4M3 codes of x / (1/32)."""
    out = torch.empty(shape, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        x = torch.randn(part.shape, generator=g, device=DEV, dtype=torch.float32)
        part.copy_((x * 32).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x)
    return out


def _tables(lens, page, width, pool, g, nothing):
    """Page tables: every sequence's pages somewhere in the pool; entries behind its last page hold `nothing`."""
    need = [-(-n // page) for n in lens]
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor(np.concatenate([[0], np.cumsum(need)[:-1]]) if need else [], dtype=torch.int64, device=DEV)
    p = torch.arange(width, device=DEV)
    t = perm[(first[:, None] + p[None]).clamp(max=pool - 1)]
    return torch.where(p[None] < torch.tensor(need, device=DEV)[:, None], t, torch.full_like(t, nothing))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _random_tree(batch, nodes, g):
    """Masks of random trees: node i sees itself and the nodes on its way to the root; a node's parent is an
    earlier node, mostly a recent one, or none. [batch, nodes, ceil(nodes / 32)] int32, bit j: sees node j."""
    u = torch.rand((batch, nodes), generator=g, device=DEV)
    i = torch.arange(nodes, device=DEV)
    parent = (i[None] - 1 - torch.floor(u * u * torch.clamp(i[None], max=12))).long()
    sees = torch.zeros((batch, nodes, nodes), dtype=torch.bool, device=DEV)
    for k in range(nodes):
        if k:
            up = parent[:, k].clamp(min=0)
            sees[:, k] = sees[torch.arange(batch, device=DEV), up] & (parent[:, k] >= 0)[:, None]
        sees[:, k, k] = True
    words = -(-nodes // 32)
    bits = torch.zeros((batch, nodes, words * 32), dtype=torch.int64, device=DEV)
    bits[:, :, :nodes] = sees
    w = (bits.view(batch, nodes, words, 32) << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    page, pool = c["page"], _pool(c)
    s = {"case": c}
    if c["op"] == "resize":
        old, new = _resize_plan(c)
        width = max(1, max(-(-n // page) for n in old + new))
        s["table"] = _tables(old, page, width, pool, g, -1)
        s["refs"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        live = s["table"][s["table"] >= 0].long()
        s["refs"][live] = 1
        s["lens"], s["new_lens"] = _i32(old), _i32(new)
        s["new_table"], s["new_refs"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        return s
    if c["op"] == "fork":
        lens, parents = _fork_plan(c)
        width = -(-max(lens) // page)
        s["table"] = _tables(lens, page, width, pool, g, -1)
        s["refs"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        s["k"] = _cache((c["layers"], pool, page, c["hk"], D), c["fp8"], g)
        s["v"] = _cache((c["layers"], pool, page, c["hk"], D), c["fp8"], g)
        s["lens"], s["parents"] = _i32(lens), _i32(parents)
        s["new_table"] = torch.empty((c["children"], width), dtype=torch.int32, device=DEV)
        s["new_refs"] = torch.empty_like(s["refs"])
        s["new_lens"] = torch.empty(c["children"], dtype=torch.int32, device=DEV)
        return s
    least = c["nodes"] if c["op"] == "tree" else c["tokens"]
    lens, cnt = _lens(c, least), _counts(c, least)
    width = -(-c["kv"] // page)
    s["lens"], s["counts"] = _i32(lens), (_i32(cnt) if c["ragged"] else None)
    s["table"] = _tables(lens, page, width, pool, g, 1 << 30)
    if c["op"] == "tree":
        s["k"] = _cache((pool, page, c["hk"], D), c["fp8"], g)
        s["v"] = _cache((pool, page, c["hk"], D), c["fp8"], g)
        s["q"] = torch.randn((c["batch"], c["nodes"], c["hq"], D), generator=g, device=DEV).to(torch.bfloat16)
        s["mask"] = _random_tree(c["batch"], c["nodes"], g) if c["tree"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((c["batch"], c["nodes"], c["hq"]), dtype=torch.float32, device=DEV)
    elif c["op"] == "append":
        s["k"] = _cache((pool, page, c["hk"], D), c["fp8"], g)
        s["v"] = _cache((pool, page, c["hk"], D), c["fp8"], g)
        # the projections' output: query, key and value heads of a token side by side
        qkv = torch.randn((c["batch"], c["tokens"], c["hq"] + 2 * c["hk"], D), generator=g, device=DEV).to(torch.bfloat16)
        s["k_new"], s["v_new"] = qkv[:, :, c["hq"]:c["hq"] + c["hk"]], qkv[:, :, c["hq"] + c["hk"]:]
    else:
        s["k"] = _cache((c["layers"], pool, page, c["hk"], D), c["fp8"], g)
        s["v"] = _cache((c["layers"], pool, page, c["hk"], D), c["fp8"], g)
        score = torch.rand((c["batch"], c["tokens"]), generator=g, device=DEV)
        score = score.masked_fill(torch.arange(c["tokens"], device=DEV)[None] >= _i32(cnt)[:, None], 2.0)
        acc = score.argsort(dim=1)[:, :c["accept"]]
        n = _i32([min(c["accept"], t) for t in cnt])
        big = acc.masked_fill(torch.arange(c["accept"], device=DEV)[None] >= n[:, None], 1 << 20).sort(dim=1)[0]
        s["accepted"] = big.masked_fill(big == 1 << 20, -1).to(torch.int32)
        s["n_accepted"] = n
        s["new_lens"] = torch.empty_like(n)
    return s


# -------------------------------------------------------------- the plain forms

def _rows(pages, table, page):
    """[batch, positions, heads, 512] of the cached rows, by a table whose entries may be out of range."""
    idx = table.long().clamp(0, pages.shape[0] - 1)
    x = pages[idx]
    return x.reshape(table.shape[0], table.shape[1] * page, *pages.shape[2:])


def _seen(mask, nodes, cnt):
    """[batch, nodes, nodes]: node i sees node j (of those that there are)."""
    j = torch.arange(nodes, device=DEV)
    if mask is None:
        s = (j[None, :] <= j[:, None])[None].expand(cnt.shape[0], nodes, nodes)
    else:
        s = ((mask[:, :, j >> 5] >> (j & 31)) & 1) == 1
    return s & (j[None, None] < cnt[:, None, None])


def _tree_plain(s):
    c = s["case"]
    q, table, page = s["q"], s["table"], c["page"]
    b, t, hq, _ = q.shape
    hk, g = c["hk"], hq // c["hk"]
    lens = s["lens"].long()
    cnt = torch.full_like(lens, t) if s["counts"] is None else s["counts"].long()
    start = lens - cnt
    n = table.shape[1] * page
    j = torch.arange(n, device=DEV)
    i = torch.arange(t, device=DEV)
    seen = _seen(s["mask"], t, cnt)
    depth = seen.sum(-1) - 1
    node = (j[None] - start[:, None])
    drafted = node >= 0
    at = node.clamp(0, t - 1)
    where = torch.where(drafted, start[:, None] + depth.gather(1, at), j[None])
    here = start[:, None] + depth
    vis = ~drafted[:, None, :] | seen.gather(2, at[:, None, :].expand(b, t, n))
    live = j[None] < lens[:, None]
    vis = vis & live[:, None]
    if c["window"] > 0:
        vis = vis & ((where[:, None] > here[:, :, None] - c["window"]) | (where[:, None] < c["sinks"]))
    vis = vis & ((i[None] < cnt[:, None]) & (start[:, None] + i[None] >= 0))[:, :, None]

    def rows(pages):
        x = _rows(pages, table, page)
        x = x.view(torch.float8_e4m3fn).float() / 32 if c["fp8"] else x.float()
        return torch.where(live[:, :, None, None], x, torch.zeros_like(x)).permute(0, 2, 1, 3)

    qf = q.float().reshape(b, t, hk, g, D).permute(0, 2, 1, 3, 4).reshape(b, hk, t * g, D)
    x = torch.matmul(qf, rows(s["k"]).transpose(2, 3)) * D ** -0.5
    x = x.masked_fill(~vis[:, None, :, None].expand(b, 1, t, g, n).reshape(b, 1, t * g, n), NEG)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == NEG, torch.zeros_like(m), m)
    p = torch.exp(x - m0)
    del x
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows(s["v"])) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m0 + torch.log(torch.where(l > 0, l, torch.ones_like(l))), torch.full_like(l, NEG))
    s["out"].copy_(o.view(b, hk, t, g, D).permute(0, 2, 1, 3, 4).reshape(b, t, hq, D))
    s["lse"].copy_(lse.view(b, hk, t, g).permute(0, 2, 1, 3).reshape(b, t, hq))
    return s["out"], s["lse"]


def _places(s, tokens):
    """(sequence, token) of each new token that there is, and its page and slot."""
    page, lens = s["case"]["page"], s["lens"].long()
    cnt = torch.full_like(lens, tokens) if s["counts"] is None else s["counts"].long()
    t = torch.arange(tokens, device=DEV)
    b, t = torch.nonzero(t[None] < cnt[:, None], as_tuple=True)
    pos = (lens - cnt)[b] + t
    return b, t, s["table"].long()[b, pos // page], pos % page


def _append_plain(s):
    c = s["case"]
    b, t, pg, slot = _places(s, c["tokens"])
    for new, pages in ((s["k_new"], s["k"]), (s["v_new"], s["v"])):
        x = new[b, t]
        if c["fp8"]:
            x = (x.float() / 0.03125).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pages[pg, slot] = x
    return s["k"], s["v"]


def _compact_plain(s):
    c, page, lens = s["case"], s["case"]["page"], s["lens"].long()
    cnt = torch.full_like(lens, c["tokens"]) if s["counts"] is None else s["counts"].long()
    start = lens - cnt
    i = torch.arange(c["accept"], device=DEV)
    b, i = torch.nonzero(i[None] < s["n_accepted"][:, None], as_tuple=True)
    src, dst = start[b] + s["accepted"].long()[b, i], start[b] + i
    table = s["table"].long()
    for pages in (s["k"], s["v"]):
        pages[:, table[b, dst // page], dst % page] = pages[:, table[b, src // page], src % page]
    s["new_lens"].copy_(start + s["n_accepted"])
    return s["k"], s["v"], s["new_lens"]


def _held(lens, page, width):
    return torch.arange(width, device=DEV)[None] < ((lens.long() + page - 1) // page)[:, None]


def _fork_plain(s):
    c, page, table = s["case"], s["case"]["page"], s["table"].long()
    lens, parents = s["lens"].long(), s["parents"].long()
    n, width = lens[parents], table.shape[1]
    kids = parents.shape[0]
    new = torch.where(_held(n, page, width), table[parents], torch.full_like(table[parents], -1))
    k = torch.arange(kids, device=DEV)
    older = ((parents[None] == parents[:, None]) & (k[None] < k[:, None])).any(1)
    copies = older & (n % page != 0)
    refs = s["refs"].clone()
    refs.index_add_(0, table[_held(lens, page, width)], torch.full_like(table[_held(lens, page, width)], -1, dtype=torch.int32))
    last = (n // page).clamp(max=width - 1)
    shared = _held(n, page, width) & ~(copies[:, None] & (torch.arange(width, device=DEV)[None] == last[:, None]))
    refs.index_add_(0, new[shared], torch.ones_like(new[shared], dtype=torch.int32))
    who = torch.nonzero(copies)[:, 0]
    fresh = torch.nonzero(refs == 0)[:, 0][:who.shape[0]]
    src = new[who, last[who]]
    new[who, last[who]] = fresh
    refs[fresh] = 1
    live = torch.arange(page, device=DEV)[None] < (n % page)[who][:, None]
    w, slot = torch.nonzero(live, as_tuple=True)
    for pages in (s["k"], s["v"]):
        pages[:, fresh[w], slot] = pages[:, src[w], slot]
    s["new_table"].copy_(new)
    s["new_lens"].copy_(n)
    s["new_refs"].copy_(refs)
    return s["k"], s["v"], s["new_table"], s["new_lens"], s["new_refs"]


def _resize_plain(s):
    page, table, width = s["case"]["page"], s["table"].long(), s["table"].shape[1]
    a, z = _held(s["lens"], page, width), _held(s["new_lens"], page, width)
    refs = s["refs"].clone()
    gone = table[a & ~z]
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    b, p = torch.nonzero(z & ~a, as_tuple=True)
    fresh = torch.nonzero(refs == 0)[:, 0][:b.shape[0]]
    new = torch.where(a & z, table, torch.full_like(table, -1))
    new[b, p] = fresh
    refs[fresh] = 1
    s["new_table"].copy_(new)
    s["new_refs"].copy_(refs)
    return s["new_table"], s["new_refs"]


# ------------------------------------------------------------------ one pass

def _bits(pages, fp8):
    """Moved rows as whole numbers (they have to be equal)."""
    return pages if fp8 else pages.view(torch.int16)


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s)
    if c["op"] == "tree":
        return _tree_plain(s)
    if c["op"] == "append":
        k, v = _append_plain(s)
        return _written(k, v, c)
    if c["op"] == "compact":
        k, v, n = _compact_plain(s)
        return _bits(k, c["fp8"]), _bits(v, c["fp8"]), n
    if c["op"] == "fork":
        k, v, t, n, r = _fork_plain(s)
        return _bits(k, c["fp8"]), _bits(v, c["fp8"]), t, n, r
    return _resize_plain(s)


def _written(k, v, c):
    """The caches after an append: E4M3 codes as the type that says what they stand for, bf16 as whole numbers."""
    return (k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)) if c["fp8"] else (_bits(k, False), _bits(v, False))


def _run_own(s):
    import head_dim_flashattention_gb300 as fa
    c = s["case"]
    if c["op"] == "tree":
        if c["fp8"]:
            return fa.fa512_decode_paged_tree_fp8(s["q"], s["k"], s["v"], s["table"], s["lens"], s["mask"], s["out"],
                                                  s["lse"], q_lens=s["counts"], k_scale=1 / 32, v_scale=1 / 32,
                                                  max_kv_len=c["kv"], window=c["window"], n_sinks=c["sinks"])
        return fa.fa512_decode_paged_tree(s["q"], s["k"], s["v"], s["table"], s["lens"], s["mask"], s["out"], s["lse"],
                                          q_lens=s["counts"], max_kv_len=c["kv"], window=c["window"],
                                          n_sinks=c["sinks"])
    if c["op"] == "append":
        if c["fp8"]:
            fa.fa512_cache_append_fp8(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"],
                                      q_lens=s["counts"], k_scale=1 / 32, v_scale=1 / 32)
        else:
            fa.fa512_cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], q_lens=s["counts"])
        return _written(s["k"], s["v"], c)
    if c["op"] == "compact":
        fa.fa512_cache_compact(s["k"], s["v"], s["table"], s["lens"], s["accepted"], s["n_accepted"], s["new_lens"],
                               q_len=c["tokens"], q_lens=s["counts"])
        return _bits(s["k"], c["fp8"]), _bits(s["v"], c["fp8"]), s["new_lens"]
    if c["op"] == "fork":
        fa.fa512_cache_fork(s["k"], s["v"], s["table"], s["lens"], s["parents"], s["refs"], s["new_table"],
                            s["new_lens"], s["new_refs"])
        return _bits(s["k"], c["fp8"]), _bits(s["v"], c["fp8"]), s["new_table"], s["new_lens"], s["new_refs"]
    return fa.fa512_cache_resize(s["table"], s["lens"], s["new_lens"], s["refs"], s["new_table"], s["new_refs"],
                                 page_size=c["page"])


# ------------------------------------------------------------- 64-bit outputs

def exact(case, seed):
    """The attention from its definition, one sequence and KV head at a time, and the E4M3 values by searching the
    256 codes' values. What is only moved has no value of its own here."""
    c = case
    if c["op"] == "append" and c["fp8"]:
        s = prepare(case, seed)
        codes = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
        middle = (codes[1:] + codes[:-1]) / 2
        got = []
        for new, pages in ((s["k_new"], s["k"]), (s["v_new"], s["v"])):
            want = pages.view(torch.float8_e4m3fn).float()
            for b, (n, t) in enumerate(zip(_lens(c, c["tokens"]), _counts(c, c["tokens"]))):
                x = new[b, :t].double() * 32
                up, down = torch.bucketize(x.abs(), middle, right=True), torch.bucketize(x.abs(), middle)
                k = torch.where(up % 2 == 0, up, down)  # a tie goes to the even code
                pos = torch.arange(n - t, n, device=DEV)
                want[s["table"][b].long()[pos // c["page"]], pos % c["page"]] = (codes[k] * torch.sign(x)).float()
            got.append(want.double())
        return tuple(got)
    if c["op"] != "tree":
        return None
    s = prepare(case, seed)
    b, t, hq, _ = s["q"].shape
    g, page = hq // c["hk"], c["page"]
    out = torch.zeros((b, t, hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((b, t, hq), NEG, dtype=torch.float64, device=DEV)
    masks = None if s["mask"] is None else s["mask"].cpu().numpy().astype(np.int64) & 0xFFFFFFFF
    for i, (n, cnt) in enumerate(zip(_lens(c, t), _counts(c, t))):
        first = n - cnt
        sees = np.tril(np.ones((cnt, cnt), bool))
        if masks is not None:
            sees = np.array([[bool(masks[i, a, z // 32] >> (z % 32) & 1) for z in range(cnt)] for a in range(cnt)])
        depth = sees.sum(1) - 1
        place = np.concatenate([np.arange(first), first + depth])
        ok = np.concatenate([np.ones((cnt, first), bool), sees], axis=1)
        if c["window"]:
            ok &= (place[None] > (first + depth)[:, None] - c["window"]) | (place[None] < c["sinks"])
        ok = torch.from_numpy(ok).to(DEV)
        keep = torch.nonzero(ok.any(0))[:, 0]
        if not keep.numel():
            continue
        ok = ok[:, keep]
        pg, slot = s["table"][i].long()[keep // page], keep % page
        for h in range(c["hk"]):
            kk, vv = s["k"][pg, slot, h], s["v"][pg, slot, h]
            if c["fp8"]:
                kk, vv = kk.view(torch.float8_e4m3fn).double() / 32, vv.view(torch.float8_e4m3fn).double() / 32
            kk, vv = kk.double(), vv.double()
            qq = s["q"][i, :cnt, h * g:(h + 1) * g].double()
            x = torch.einsum("tgd,nd->tgn", qq, kk) / math.sqrt(D)
            x = torch.where(ok[:, None], x, torch.full_like(x, NEG))
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(z == NEG, torch.zeros_like(z), z)[..., None])
            out[i, :cnt, h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", p, vv)
            lse[i, :cnt, h * g:(h + 1) * g] = z
    return out, lse
