"""Cases of decoding that reads less of a long cache.

Five operators, used one after another by a program that serves long contexts
over a paged cache of heads of 512 dimensions:

  append   writes the new tokens' keys and values into a cache of 4 bits an
           element: a row of a head is 256 bytes of E2M1 codes (element 2 i in
           the low half of byte i) and 32 E4M3 scales, one for 16 elements; an
           element is tensor scale * group scale * code
  decode   attention of the newest token(s) of each sequence over such a cache
  bounds   the smallest and largest key element of each channel of the pages
           that were written to
  select   the pages whose bounds allow the largest product with the queries,
           for each sequence and KV head; the first and last pages always
  sparse   attention over the selected pages alone, over a cache in bf16, in
           E4M3 or in 4 bits

Each has a plain form here in elementary torch operations.
"""
import math
import random

import numpy as np
import torch

own = False

D = 512
ROW4 = 288          # bytes of a row of one head in 4 bits: codes, then scales
DEV = "cuda"
NEG = float("-inf")
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
BYTES = {"bf16": 1024, "e4m3": 512, "e2m1": ROW4}
# tensor scales of keys and values: what a calibration leaves (powers of two)
KS, VS = 0.5, 2.0


# ------------------------------------------------------------------- the cases

def listed():
    """Sizes: 8 query heads over 4 KV heads, pages of 64, caches of 4,096, 16,384
    and 28,672 positions and batches of 1, 16 and 64 are the decode workloads of
    this repository; 32 over 4 are its prefill head counts."""
    return [
        # one decode step's token of each sequence goes into the 4-bit cache
        {"name": "append_b16_t1", "op": "append", "batch": 16, "tokens": 1, "hq": 8, "hk": 4, "kv": 4096, "page": 64,
         "ragged": False},
        # prompt pieces of a batch
        {"name": "append_b8_t4096", "op": "append", "batch": 8, "tokens": 4096, "hq": 32, "hk": 4, "kv": 16384,
         "page": 64, "ragged": True},
        # one user: the step's latency counts
        {"name": "decode_b1_kv4096", "op": "decode", "batch": 1, "tokens": 1, "hq": 8, "hk": 4, "kv": 4096, "page": 64,
         "window": 0, "ragged": False},
        # drafts of four tokens over contexts of different lengths
        {"name": "decode_b16_t4_kv16384", "op": "decode", "batch": 16, "tokens": 4, "hq": 8, "hk": 4, "kv": 16384,
         "page": 64, "window": 0, "ragged": True},
        # the whole server: as many long contexts as there are
        {"name": "decode_b64_kv28672", "op": "decode", "batch": 64, "tokens": 1, "hq": 8, "hk": 4, "kv": 28672,
         "page": 64, "window": 0, "ragged": False},
        # after each decode step: the page that is filling
        {"name": "bounds_b16_t1", "op": "bounds", "batch": 16, "tokens": 1, "hk": 4, "kv": 4096, "page": 64,
         "kind": "bf16", "ragged": False},
        # after a prompt's pieces
        {"name": "bounds_fp4_b8_t4096", "op": "bounds", "batch": 8, "tokens": 4096, "hk": 4, "kv": 16384, "page": 64,
         "kind": "e2m1", "ragged": True},
        # one user's long context
        {"name": "select_b1_kv28672", "op": "select", "batch": 1, "tokens": 1, "hq": 8, "hk": 4, "kv": 28672,
         "page": 64, "pick": 64, "first": 1, "last": 4, "ragged": False},
        # many of them
        {"name": "select_b64_kv28672", "op": "select", "batch": 64, "tokens": 1, "hq": 8, "hk": 4, "kv": 28672,
         "page": 64, "pick": 64, "first": 1, "last": 4, "ragged": True},
        # one user: 64 of 448 pages
        {"name": "sparse_b1_n64", "op": "sparse", "batch": 1, "tokens": 1, "hq": 8, "hk": 4, "kv": 28672, "page": 64,
         "pick": 64, "kind": "bf16", "ragged": False},
        # many users, small pages, 8-bit cache, 8 query heads a KV head
        {"name": "sparse_fp8_b16_n200", "op": "sparse", "batch": 16, "tokens": 1, "hq": 32, "hk": 4, "kv": 16384,
         "page": 16, "pick": 200, "kind": "e4m3", "ragged": True},
        # the whole server over the 4-bit cache
        {"name": "sparse_fp4_b64_n64", "op": "sparse", "batch": 64, "tokens": 1, "hq": 8, "hk": 4, "kv": 28672,
         "page": 64, "pick": 64, "kind": "e2m1", "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "bounds", "select", "sparse", "sparse"])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    hq, hk = rng.choice([(8, 4), (8, 4), (32, 4), (16, 1), (12, 4), (4, 4), (8, 1)])
    tokens = 1 if rng.random() < 0.5 else rng.randint(1, 16 // (hq // hk))
    c = {"op": op, "batch": _log(rng, 1, 64), "tokens": tokens, "hq": hq, "hk": hk, "kv": _log(rng, 130, 28672),
         "page": page, "ragged": rng.random() < 0.5}
    if op == "append" or op == "bounds":
        c["tokens"] = _log(rng, 1, 4096)
        c["kv"] = c["tokens"] + _log(rng, 1, 4096)
    if op == "decode":
        c["window"] = _log(rng, 1, 8192) if rng.random() < 0.4 else 0
    if op == "bounds" or op == "sparse":
        c["kind"] = rng.choice(["bf16", "e4m3", "e2m1"])
    if op == "select" or op == "sparse":
        c["pick"] = _log(rng, 6, max(6, 8192 // page))
    if op == "select":
        c["first"], c["last"] = rng.randint(0, 2), rng.randint(1, 4)
    most = [work(x) for x in listed() if x["op"] == op]
    top = max(w["bytes"] for w in most)
    while c["batch"] > 1 and (work(c)["bytes"] > top or work(c)["flops"] > 64 * top):
        c["batch"] = (c["batch"] + 1) // 2
    while c["op"] in ("append", "bounds") and work(c)["bytes"] > top:
        c["tokens"] = (c["tokens"] + 1) // 2
    return c


# ------------------------------------------------- lengths and work of one case

def _lens(c):
    """The lengths of the sequences, from the case alone."""
    kv, b = c["kv"], c["batch"]
    if not c["ragged"]:
        return [kv] * b
    return [max(min(kv, c["tokens"]), kv - (i * 7919 + 13) % max(1, kv // 2)) for i in range(b)]


def _counts(c):
    """How many new tokens each sequence has, of the most."""
    if not c["ragged"] or c["op"] not in ("append", "bounds"):
        return [c["tokens"]] * c["batch"]
    return [max(1, c["tokens"] - (i * 31) % max(1, (c["tokens"] + 1) // 2)) for i in range(c["batch"])]


def work(case):
    c, page = case, case["page"]
    lens, cnt = _lens(c), _counts(c)
    if c["op"] == "append":
        return {"bytes": sum(cnt) * c["hk"] * 2 * (1024 + ROW4), "flops": 0}
    if c["op"] == "bounds":
        b = 0
        for n, t in zip(lens, cnt):
            p0, p1 = (n - t) // page, (n - 1) // page
            b += (n - p0 * page) * c["hk"] * BYTES[c["kind"]] + (p1 - p0 + 1) * c["hk"] * 2048
        return {"bytes": b, "flops": 0}
    rows = c["tokens"] * c["hq"]
    if c["op"] == "select":
        pages = sum(-(-n // page) for n in lens)
        return {"bytes": pages * (c["hk"] * 2048 + 4) + c["batch"] * (rows * 1024 + c["hk"] * c["pick"] * 4),
                "flops": pages * rows * D * 4}
    row, b, f = BYTES[c.get("kind", "e2m1")], 0, 0
    for n in lens:
        if c["op"] == "decode":
            seen = n if not c["window"] else min(n, c["window"] + c["tokens"] - 1)
            pairs = n if not c["window"] else min(n, c["window"])
        else:
            # the last page, which is partly filled, is always among them
            seen = pairs = min(n, (c["pick"] - 1) * page + (n - 1) % page + 1)
            b += c["hk"] * min(c["pick"], -(-n // page)) * 4
        b += seen * c["hk"] * row * 2 + rows * 2048
        f += pairs * rows * D * 4
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------- the inputs

def _pool(c):
    """Pages of the pool."""
    return c["batch"] * -(-c["kv"] // c["page"]) + 8


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _cache(rows, kind, scale, g):
    """Cached rows [*rows, bytes or elements] as a model leaves them: roughly normal values with channels of
    different size, in the format of the cache."""
    n = math.prod(rows)
    shape = (n, D) if kind != "e2m1" else (n, ROW4)
    out = torch.empty(shape, dtype=torch.bfloat16 if kind == "bf16" else torch.uint8, device=DEV)
    size = torch.exp(torch.randn(D, generator=g, device=DEV) * 0.4)
    for i in range(0, n, 1 << 18):
        part = out[i:i + (1 << 18)]
        x = torch.randn((part.shape[0], D), generator=g, device=DEV) * size
        if kind == "bf16":
            part.copy_(x)
        elif kind == "e4m3":
            part.copy_((x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            codes, s = _to_4bit(x.to(torch.bfloat16).float(), scale)
            part[:, :256] = codes
            part[:, 256:] = s
    return out.view(*rows, shape[1])


def _tables(lens, page, width, pool, g, nothing):
    """Page tables: every sequence's pages somewhere in the pool; entries behind its last page hold `nothing`."""
    need = [-(-n // page) for n in lens]
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor(np.concatenate([[0], np.cumsum(need)[:-1]]), dtype=torch.int64, device=DEV)
    p = torch.arange(width, device=DEV)
    t = perm[(first[:, None] + p[None]).clamp(max=pool - 1)]
    return torch.where(p[None] < torch.tensor(need, device=DEV)[:, None], t, torch.full_like(t, nothing))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    page, pool, hk = c["page"], _pool(c), c["hk"]
    lens = _lens(c)
    width = -(-c["kv"] // page)
    s = {"case": c, "lens": _i32(lens), "counts": _i32(_counts(c)) if c["ragged"] else None,
         "table": _tables(lens, page, width, pool, g, 1 << 30)}
    if c["op"] in ("decode", "select", "sparse"):
        s["q"] = torch.randn((c["batch"], c["tokens"], c["hq"], D), generator=g, device=DEV).to(torch.bfloat16)
    if c["op"] in ("decode", "sparse"):
        kind = c.get("kind", "e2m1")
        s["k"], s["v"] = _cache((pool, page, hk), kind, KS, g), _cache((pool, page, hk), kind, VS, g)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:3], dtype=torch.float32, device=DEV)
    if c["op"] == "append":
        s["k"], s["v"] = _cache((pool, page, hk), "e2m1", KS, g), _cache((pool, page, hk), "e2m1", VS, g)
        # the projections' output: query, key and value heads of a token side by side
        qkv = torch.randn((c["batch"], c["tokens"], c["hq"] + 2 * hk, D), generator=g, device=DEV).to(torch.bfloat16)
        s["k_new"], s["v_new"] = qkv[:, :, c["hq"]:c["hq"] + hk], qkv[:, :, c["hq"] + hk:]
    if c["op"] == "bounds":
        s["k"] = _cache((pool, page, hk), c["kind"], KS, g)
        s["bounds"] = torch.zeros((pool, hk, 2, D), dtype=torch.bfloat16, device=DEV)
    if c["op"] == "select":
        # bounds of keys that vary around their page's mean
        mid = torch.randn((pool, hk, D), generator=g, device=DEV) * 0.4
        wide = 2.0 + 0.6 * torch.rand((pool, hk, 2, D), generator=g, device=DEV)
        s["bounds"] = torch.stack([mid - wide[:, :, 0], mid + wide[:, :, 1]], 2).to(torch.bfloat16)
        s["pages"] = torch.empty((c["batch"], hk, c["pick"]), dtype=torch.int32, device=DEV)
    if c["op"] == "sparse":
        # some pages of each sequence, the last one among them, in rising order
        r = torch.rand((c["batch"], hk, width), generator=g, device=DEV)
        held = (s["lens"].long() + page - 1) // page
        p = torch.arange(width, device=DEV)
        r = r.masked_fill(p == (held - 1)[:, None, None], 2.0).masked_fill(p >= held[:, None, None], -1.0)
        n = min(c["pick"], width)
        at = r.argsort(dim=-1, descending=True)[..., :n]
        at = at.masked_fill(at >= held[:, None, None], 1 << 30).sort(dim=-1)[0]
        s["pages"] = torch.full((c["batch"], hk, c["pick"]), -1, dtype=torch.int32, device=DEV)
        s["pages"][..., :n] = at.masked_fill(at == 1 << 30, -1).to(torch.int32)
    return s


# -------------------------------------------------------------- the plain forms

def _to_4bit(x, scale):
    """Codes [n, 256] and scale bytes [n, 32] of rows x [n, 512] in 32 bits: the scale is the E4M3 value nearest to a
    sixth of the group's largest magnitude, a code the E2M1 value nearest to the quotient, both ties to even."""
    y = (x / scale).view(-1, 32, 16)
    s = (y.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    z = torch.where(sf > 0, y / sf, torch.zeros_like(y))
    middle = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    up, down = torch.bucketize(z.abs(), middle, right=True), torch.bucketize(z.abs(), middle)
    code = torch.where(up % 2 == 0, up, down)      # they differ in a tie, which goes to the even code
    code = (code | torch.where(torch.signbit(z), 8, 0)).to(torch.uint8).view(-1, 256, 2)
    return code[..., 0] | (code[..., 1] << 4), s.view(torch.uint8)


def _from_4bit(rows):
    """Rows [..., 288] -> [..., 512] in 32 bits, without the tensor scale."""
    half = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float32, device=rows.device)
    two = torch.stack([half.repeat(16), half.repeat_interleave(16)], -1)      # of a byte: low half, high half
    x = two[rows[..., :256].int()].flatten(-2)
    s = rows[..., 256:].contiguous().view(torch.float8_e4m3fn).float()
    return x.view(*s.shape, 16).mul_(s[..., None]).flatten(-2)


def _values(rows, kind):
    """Cached rows in 32 bits, without the tensor scale."""
    return _from_4bit(rows) if kind == "e2m1" else (rows.view(torch.float8_e4m3fn) if kind == "e4m3" else rows).float()


def _scales(kind):
    return (1.0, 1.0) if kind == "bf16" else (KS, VS)


def _append_plain(s):
    c, page, lens = s["case"], s["case"]["page"], s["lens"].long()
    cnt = torch.full_like(lens, c["tokens"]) if s["counts"] is None else s["counts"].long()
    t = torch.arange(c["tokens"], device=DEV)
    b, t = torch.nonzero(t[None] < cnt[:, None], as_tuple=True)
    pos = (lens - cnt)[b] + t
    pg, slot = s["table"].long()[b, pos // page], pos % page
    for new, pages, scale in ((s["k_new"], s["k"], KS), (s["v_new"], s["v"], VS)):
        codes, by = _to_4bit(new[b, t].float().view(-1, D), scale)
        pages[pg, slot] = torch.cat([codes, by], -1).view(-1, c["hk"], ROW4)
    return s["k"], s["v"]


def _softmax(s, x, vis, values):
    """x [b, hk, rows, n] scores, vis the same shape or broadcast, values [b, hk, n, 512] -> out, lse of the state."""
    b, t, hq, _ = s["q"].shape
    hk = x.shape[1]
    x = x.masked_fill(~vis, NEG)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == NEG, torch.zeros_like(m), m)
    p = torch.exp(x - m0)
    del x
    l = p.sum(-1, keepdim=True)
    some = torch.where(l > 0, l, torch.ones_like(l))
    o = torch.matmul(p, values) / some
    lse = torch.where(l > 0, m0 + torch.log(some), torch.full_like(l, NEG))
    s["out"].copy_(o.view(b, hk, t, hq // hk, D).permute(0, 2, 1, 3, 4).reshape(b, t, hq, D))
    s["lse"].copy_(lse.view(b, hk, t, hq // hk).permute(0, 2, 1, 3).reshape(b, t, hq))
    return s["out"], s["lse"]


def _queries(s):
    """[b, hk, tokens * group, 512] in 32 bits."""
    b, t, hq, _ = s["q"].shape
    hk = s["case"]["hk"]
    return s["q"].float().reshape(b, t, hk, hq // hk, D).permute(0, 2, 1, 3, 4).reshape(b, hk, t * hq // hk, D)


def _decode_plain(s):
    c, page, lens = s["case"], s["case"]["page"], s["lens"].long()
    b, t, hq, _ = s["q"].shape
    hk, n = c["hk"], s["table"].shape[1] * page
    at = s["table"].long().clamp(0, s["k"].shape[0] - 1)
    j = torch.arange(n, device=DEV)
    live = j[None] < lens[:, None]
    pos = (lens - t)[:, None] + torch.arange(t, device=DEV)[None]
    vis = (j[None, None] <= pos[..., None]) & live[:, None]
    if c["window"] > 0:
        vis &= j[None, None] > pos[..., None] - c["window"]

    def rows(pages):
        x = _from_4bit(pages[at].view(b, n, hk, ROW4)).masked_fill_(~live[:, :, None, None], 0.0)
        return x.permute(0, 2, 1, 3)

    x = torch.matmul(_queries(s), rows(s["k"]).transpose(2, 3)) * (KS * D ** -0.5)
    return _softmax(s, x, vis[:, None, :, None].expand(b, 1, t, hq // hk, n).reshape(b, 1, t * hq // hk, n),
                    rows(s["v"]).mul_(VS))


def _bounds_plain(s):
    c, page, lens = s["case"], s["case"]["page"], s["lens"].long()
    cnt = torch.full_like(lens, c["tokens"]) if s["counts"] is None else s["counts"].long()
    p = torch.arange(s["table"].shape[1], device=DEV)
    b, p = torch.nonzero((p >= ((lens - cnt) // page)[:, None]) & (p <= ((lens - 1) // page)[:, None]), as_tuple=True)
    pg = s["table"].long()[b, p]
    x = _values(s["k"][pg], c["kind"])                                       # [n, page, hk, 512]
    live = (p * page)[:, None] + torch.arange(page, device=DEV) < lens[b][:, None]
    live = live[:, :, None, None]
    s["bounds"][pg, :, 0] = x.masked_fill(~live, math.inf).amin(1).to(torch.bfloat16)
    s["bounds"][pg, :, 1] = x.masked_fill(~live, NEG).amax(1).to(torch.bfloat16)
    return s["bounds"]


def _select_plain(s):
    """The score of a page is the largest, over the rows of the KV head, of sum_d max(q_d lo_d, q_d hi_d). The order of
    that sum in 32 bits is part of the operator, so that scores next to the border fall the same way everywhere:
    channels c and c + 256, then the eight of c // 8 by halves, then the 32 groups by halves."""
    c, page, lens = s["case"], s["case"]["page"], s["lens"].long()
    b, hk, n = lens.shape[0], c["hk"], s["table"].shape[1]
    at = s["table"].long().clamp(0, s["bounds"].shape[0] - 1)
    bounds = s["bounds"][at].float().permute(0, 2, 1, 3, 4)                  # [b, hk, pages, 2, 512]
    q = _queries(s)[:, :, :, None]                                           # [b, hk, rows, 1, 512]
    x = torch.maximum(q * bounds[:, :, None, :, 0], q * bounds[:, :, None, :, 1])
    x = x.view(*x.shape[:-1], 2, 32, 8).transpose(-1, -2).flatten(-3)
    while x.shape[-1] > 1:
        x = x[..., :x.shape[-1] // 2] + x[..., x.shape[-1] // 2:]
    score = x[..., 0].amax(2)                                                # [b, hk, pages]
    p = torch.arange(n, device=DEV)
    held = ((lens + page - 1) // page)[:, None, None]
    score = score.masked_fill((p < c["first"]) | (p >= held - c["last"]), math.inf).masked_fill(p >= held, NEG)
    k = min(n, c["pick"])
    best = score.sort(dim=-1, descending=True, stable=True)[1][..., :k]
    best = best.masked_fill(best >= held, 1 << 30).sort(dim=-1)[0]
    s["pages"].fill_(-1)
    s["pages"][..., :k] = best.masked_fill(best == 1 << 30, -1).to(torch.int32)
    return s["pages"]


def _sparse_plain(s):
    c, page, lens = s["case"], s["case"]["page"], s["lens"].long()
    b, t, hq, _ = s["q"].shape
    hk, n = c["hk"], c["pick"] * page
    ks, vs = _scales(c["kind"])
    pages = s["pages"].long()                                                # [b, hk, pick]
    at = s["table"].long().gather(1, pages.clamp(min=0).view(b, -1)).view(b, hk, -1).clamp(0, s["k"].shape[0] - 1)
    j = (pages[..., None] * page + torch.arange(page, device=DEV)).view(b, hk, n)
    live = (pages >= 0)[..., None].expand(b, hk, -1, page).reshape(b, hk, n) & (j < lens[:, None, None])
    pos = (lens - t)[:, None] + torch.arange(t, device=DEV)[None]
    vis = (j[:, :, None] <= pos[:, None, :, None]) & live[:, :, None]
    head = torch.arange(hk, device=DEV)[None, :, None, None]
    slot = torch.arange(page, device=DEV)

    def rows(cache):
        x = _values(cache[at[..., None], slot, head], c["kind"]).view(b, hk, n, D)
        return x.masked_fill_(~live[..., None], 0.0)

    x = torch.matmul(_queries(s), rows(s["k"]).transpose(2, 3)) * (ks * D ** -0.5)
    return _softmax(s, x, vis[:, :, :, None].expand(b, hk, t, hq // hk, n).reshape(b, hk, t * hq // hk, n),
                    rows(s["v"]).mul_(vs))


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        got = _run_own(s)
    else:
        got = {"append": _append_plain, "decode": _decode_plain, "bounds": _bounds_plain, "select": _select_plain,
               "sparse": _sparse_plain}[op](s)
    if op == "append":
        # two codes a byte, which have to be equal, and the scales as what they stand for
        return tuple(part for x in got for part in (x[..., :256], x[..., 256:].view(torch.float8_e4m3fn)))
    return got


def _run_own(s):
    import head_dim_flashattention_gb300 as fa
    c = s["case"]
    if c["op"] == "append":
        return fa.fa512_cache_append_fp4(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"],
                                         q_lens=s["counts"], k_scale=KS, v_scale=VS)
    if c["op"] == "decode":
        return fa.fa512_decode_paged_fp4(s["q"], s["k"], s["v"], s["table"], s["lens"], s["out"], s["lse"], k_scale=KS,
                                         v_scale=VS, max_kv_len=c["kv"], window=c["window"])
    if c["op"] == "bounds":
        return fa.fa512_cache_page_bounds(s["k"], s["table"], s["lens"], s["bounds"], q_len=c["tokens"],
                                          q_lens=s["counts"])
    if c["op"] == "select":
        return fa.fa512_select_pages(s["q"], s["bounds"], s["table"], s["lens"], s["pages"], page_size=c["page"],
                                     max_kv_len=c["kv"], n_first=c["first"], n_last=c["last"])
    if c["kind"] == "bf16":
        return fa.fa512_decode_paged_sparse(s["q"], s["k"], s["v"], s["table"], s["lens"], s["pages"], s["out"],
                                            s["lse"], max_kv_len=c["kv"])
    call = fa.fa512_decode_paged_sparse_fp8 if c["kind"] == "e4m3" else fa.fa512_decode_paged_sparse_fp4
    return call(s["q"], s["k"], s["v"], s["table"], s["lens"], s["pages"], s["out"], s["lse"], k_scale=KS, v_scale=VS,
                max_kv_len=c["kv"])


# ------------------------------------------------------------- 64-bit outputs

def _exact_rows(rows, kind):
    """What cached rows stand for, from the formats' definitions: sign, exponent and mantissa of each code."""
    def of(code, mant, bias, bits):
        sign = 1.0 - 2.0 * ((code >> bits) & 1).double()
        e, m = (code >> mant) & ((1 << (bits - mant)) - 1), (code & ((1 << mant) - 1)).double() / (1 << mant)
        return sign * torch.where(e == 0, m * 2.0 ** (1 - bias), (1.0 + m) * torch.exp2((e - bias).double()))
    if kind == "bf16":
        return rows.double()
    if kind == "e4m3":
        return of(rows.int(), 3, 7, 7)
    pair = rows[..., :256].int()
    code = torch.stack([pair & 15, pair >> 4], -1).flatten(-2)
    return of(code, 1, 1, 3) * of(rows[..., 256:].int(), 3, 7, 7).repeat_interleave(16, -1)


def exact(case, seed):
    """Attention from its definition, one sequence and KV head at a time; group scales by searching the E4M3 values;
    bounds of decoded keys. Codes and page numbers are whole and have no value of their own here."""
    c = case
    if c["op"] == "select":
        return None
    s = prepare(case, seed)
    page, hk, lens, cnt = c["page"], c["hk"], _lens(c), _counts(c)
    table = s["table"].long()
    if c["op"] == "append":
        grid = _exact_rows(torch.arange(127, dtype=torch.uint8, device=DEV), "e4m3")
        middle = (grid[1:] + grid[:-1]) / 2
        got = []
        for new, pages, scale in ((s["k_new"], s["k"], KS), (s["v_new"], s["v"], VS)):
            want = _exact_rows(pages[..., 256:], "e4m3")
            for b, (n, t) in enumerate(zip(lens, cnt)):
                x = new[b, :t].double() / scale
                a = x.abs().view(t, hk, 32, 16).amax(-1) / 6
                up, down = torch.bucketize(a, middle, right=True), torch.bucketize(a, middle)
                pos = torch.arange(n - t, n, device=DEV)
                want[table[b][pos // page], pos % page] = grid[torch.where(up % 2 == 0, up, down)]
            got += [None, want]
        return tuple(got)
    if c["op"] == "bounds":
        want = s["bounds"].double()
        for b, (n, t) in enumerate(zip(lens, cnt)):
            for p in range((n - t) // page, (n - 1) // page + 1):
                x = _exact_rows(s["k"][table[b, p], :min(page, n - p * page)], c["kind"])
                want[table[b, p], :, 0], want[table[b, p], :, 1] = x.amin(0), x.amax(0)
        return want
    b, t, hq, _ = s["q"].shape
    g, kind = hq // hk, c.get("kind", "e2m1")
    ks, vs = _scales(kind)
    out = torch.zeros((b, t, hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((b, t, hq), NEG, dtype=torch.float64, device=DEV)
    lists = s["pages"].cpu().numpy() if c["op"] == "sparse" else None
    for i, n in enumerate(lens):
        for h in range(hk):
            if lists is None:
                first = max(0, n - t + 1 - c["window"]) if c["window"] else 0
                j = torch.arange(first, n, device=DEV)
            else:
                some = [x for p in lists[i, h] if p >= 0 for x in range(p * page, min(n, (p + 1) * page))]
                j = torch.tensor(some, dtype=torch.int64, device=DEV)
            if not j.numel():
                continue
            pg, slot = table[i][j // page], j % page
            kk, vv = _exact_rows(s["k"][pg, slot, h], kind) * ks, _exact_rows(s["v"][pg, slot, h], kind) * vs
            pos = torch.arange(n - t, n, device=DEV)
            ok = j[None] <= pos[:, None]
            if lists is None and c["window"]:
                ok &= j[None] > pos[:, None] - c["window"]
            qq = s["q"][i, :, h * g:(h + 1) * g].double()
            x = torch.einsum("tgd,nd->tgn", qq, kk) / math.sqrt(D)
            x = torch.where(ok[:, None], x, torch.full_like(x, NEG))
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(z == NEG, torch.zeros_like(z), z)[..., None])
            out[i, :, h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", p, vv)
            lse[i, :, h * g:(h + 1) * g] = z
    return out, lse
