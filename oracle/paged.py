"""fp64 references of drafted-token attention and of the cache operations --
TEST INFRASTRUCTURE ONLY, like the rest of this package.

Plain numpy, one sequence at a time, from the operations' definitions; inputs
are torch tensors or arrays on the CPU.  bf16 and E4M3 values are widened
exactly.
"""
from __future__ import annotations

import numpy as np

from . import _bits, _i32, _u8, e4m3_table


def widen_bf16(x) -> np.ndarray:
    """bf16 tensor -> its exact values in fp64."""
    return (_bits(x).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def widen_e4m3(x) -> np.ndarray:
    """E4M3 codes -> their values in fp64."""
    return e4m3_table()[_u8(x)]


def tree_sees(tree_mask, b: int, cnt: int) -> np.ndarray:
    """[cnt, cnt] bool: token t of sequence b sees token j."""
    if tree_mask is None:
        return np.tril(np.ones((cnt, cnt), dtype=bool))
    w = _i32(tree_mask)[b].astype(np.int64) & 0xFFFFFFFF
    j = np.arange(cnt)
    return ((w[:cnt][:, j // 32] >> (j % 32)) & 1).astype(bool)


def tree_visible(tree_mask, b: int, length: int, cnt: int, window: int, n_sinks: int) -> np.ndarray:
    """[cnt, length] bool: token t of sequence b sees cached position j."""
    start = length - cnt
    sees = tree_sees(tree_mask, b, cnt)
    depth = sees.sum(axis=1) - 1
    vis = np.ones((cnt, length), dtype=bool)
    place = np.arange(length)
    for c in range(cnt):
        if start + c >= 0:
            vis[:, start + c] = sees[:, c]
            place[start + c] = start + depth[c]
    if window > 0:
        here = start + depth
        vis &= (place[None] > here[:, None] - window) | (place[None] < n_sinks)
    vis[start + np.arange(cnt) < 0] = False
    return vis


def decode_paged_tree(q, k_pages, v_pages, page_table, kv_lens, tree_mask=None, *, q_lens=None,
                      scale=None, window: int = 0, n_sinks: int = 0, k_scale=None, v_scale=None):
    """Returns ``(out, lse, weight)``: out [batch, q_len, n_q_heads, D], lse [batch, q_len, n_q_heads]
    and weight = sum_j p_j |v_j| / sum_j p_j (the scale of the rounding errors of out), all fp64.
    With k_scale / v_scale the pages hold E4M3 codes."""
    qf, pt, kl = widen_bf16(q), _i32(page_table), _i32(kv_lens)
    fp8 = k_scale is not None
    bsz, qlen, hq, d = qf.shape
    npages, psz, hk = (int(x) for x in tuple(k_pages.shape)[:3])
    G = hq // hk
    scale = d ** -0.5 if scale is None else scale
    out = np.zeros((bsz, qlen, hq, d))
    weight = np.zeros_like(out)
    lse = np.full((bsz, qlen, hq), -np.inf)
    cnts = [qlen] * bsz if q_lens is None else [int(x) for x in _i32(q_lens)]
    for b in range(bsz):
        n, cnt = int(kl[b]), cnts[b]
        vis = tree_visible(tree_mask, b, n, cnt, window, n_sinks)
        keep = np.nonzero(vis.any(axis=0))[0]
        if keep.size == 0:
            continue
        vis = vis[:, keep]
        page, slot = pt[b, keep // psz], keep % psz
        if np.any(page < 0) or np.any(page >= npages):
            raise ValueError("page table of sequence %d points outside the pool" % b)
        rows_k, rows_v = k_pages[page.astype(np.int64), slot], v_pages[page.astype(np.int64), slot]
        k = widen_e4m3(rows_k) * k_scale if fp8 else widen_bf16(rows_k)
        v = widen_e4m3(rows_v) * v_scale if fp8 else widen_bf16(rows_v)
        for h in range(hq):
            x = scale * (qf[b, :cnt, h] @ k[:, h // G].T)
            x[~vis] = -np.inf
            some = vis.any(axis=1)
            m = np.where(some, x.max(axis=1), 0.0)
            p = np.exp(x - m[:, None])
            s = np.where(some, p.sum(axis=1), 1.0)
            out[b, :cnt, h] = (p @ v[:, h // G]) / s[:, None]
            weight[b, :cnt, h] = (p @ np.abs(v[:, h // G])) / s[:, None]
            lse[b, :cnt, h] = np.where(some, m + np.log(s), -np.inf)
    return out, lse, weight


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """fp64 values -> the nearest E4M3 code (ties to even, beyond 448 to 448, NaN to NaN) as uint8."""
    x = np.asarray(x, dtype=np.float64)
    values = e4m3_table()[:127]
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.clip(np.searchsorted(values, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - values[lo], values[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def pages_of(n: int, page_size: int) -> int:
    return -(-n // page_size)


def cache_append(new, pages, page_table, kv_lens, q_lens=None, scale=None):
    """The pages (numpy: uint16 bit patterns of bf16, or uint8 codes with ``scale``) after the call."""
    bits = _bits(new)
    out = np.array(pages)
    pt, kl = _i32(page_table), _i32(kv_lens)
    bsz, qlen = bits.shape[:2]
    psz = out.shape[1]
    for b in range(bsz):
        cnt = qlen if q_lens is None else int(_i32(q_lens)[b])
        for t in range(cnt):
            pos = int(kl[b]) - cnt + t
            row = bits[b, t]
            if scale is not None:
                x = (row.astype(np.uint32) << 16).view(np.float32)
                with np.errstate(over="ignore", invalid="ignore"):
                    row = e4m3_round((x / np.float32(scale)).astype(np.float64))
            out[pt[b, pos // psz], pos % psz] = row
    return out


def cache_compact(pages, page_table, kv_lens, accepted, n_accepted, q_len: int, q_lens=None):
    """(pages [n_layers, ...] after the call, new lengths)."""
    out, pt, kl = np.array(pages), _i32(page_table), _i32(kv_lens)
    acc, na = _i32(accepted), _i32(n_accepted)
    psz = out.shape[2]
    new = np.zeros(len(kl), dtype=np.int32)
    for b in range(len(kl)):
        cnt = q_len if q_lens is None else int(_i32(q_lens)[b])
        start = int(kl[b]) - cnt
        rows = [out[:, pt[b, (start + a) // psz], (start + a) % psz].copy() for a in acc[b, :na[b]]]
        for i, r in enumerate(rows):
            out[:, pt[b, (start + i) // psz], (start + i) % psz] = r
        new[b] = start + na[b]
    return out, new


def cache_fork(k_pages, v_pages, page_table, kv_lens, parents, page_refs):
    """(k_pages, v_pages, table, lengths, counts) after the call; -1 where no page was free."""
    k, v = np.array(k_pages), np.array(v_pages)
    pt, kl, par, refs = _i32(page_table), _i32(kv_lens), _i32(parents), _i32(page_refs).copy()
    psz, width = k.shape[2], pt.shape[1]
    table = np.full((len(par), width), -1, dtype=np.int32)
    for a in range(len(kl)):
        for i in range(pages_of(int(kl[a]), psz)):
            refs[pt[a, i]] -= 1
    copies, seen = [], set()
    for c, a in enumerate(par):
        n = int(kl[a])
        for i in range(pages_of(n, psz)):
            if i == n // psz and a in seen:
                copies.append(c)
                continue
            table[c, i] = pt[a, i]
            refs[pt[a, i]] += 1
        seen.add(int(a))
    free = [int(x) for x in np.nonzero(refs == 0)[0]]
    for c, page in zip(copies, free):
        n = int(kl[par[c]])
        table[c, n // psz] = page
        refs[page] = 1
        src = pt[par[c], n // psz]
        for x in (k, v):
            x[:, page, :n % psz] = x[:, src, :n % psz]
    return k, v, table, kl[par].astype(np.int32), refs


def cache_resize(page_table, kv_lens, new_kv_lens, page_refs, page_size: int):
    """(table, counts) after the call; -1 where no page was free."""
    pt, kl, nl, refs = _i32(page_table), _i32(kv_lens), _i32(new_kv_lens), _i32(page_refs).copy()
    table = np.full_like(pt, -1)
    asked = []
    for b in range(len(kl)):
        now, then = pages_of(int(kl[b]), page_size), pages_of(int(nl[b]), page_size)
        table[b, :min(now, then)] = pt[b, :min(now, then)]
        for i in range(then, now):
            refs[pt[b, i]] -= 1
        asked += [(b, i) for i in range(now, then)]
    for (b, i), page in zip(asked, [int(x) for x in np.nonzero(refs == 0)[0]]):
        table[b, i] = page
        refs[page] = 1
    return table, refs


# ------------------------------------------------- 4-bit rows, selected pages

FP4_ROW = 288
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def widen_fp4(rows) -> np.ndarray:
    """4-bit rows [..., 288] -> the values [..., 512] they stand for without the tensor scale, in fp64."""
    r = _u8(rows)
    pairs = r[..., :256]
    code = np.stack([pairs & 15, pairs >> 4], axis=-1).reshape(*pairs.shape[:-1], 512)
    value = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    with np.errstate(invalid="ignore"):
        return value * np.repeat(e4m3_table()[r[..., 256:]], 16, axis=-1)


def fp4_rows(new, scale: float) -> np.ndarray:
    """bf16 rows [..., 512] -> 4-bit rows: fp32 quotients, each then to the nearest value, ties to even."""
    x = widen_bf16(new).astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        y = x / np.float32(scale)
        g = y.reshape(*y.shape[:-1], 32, 16)
        s8 = e4m3_round((np.max(np.abs(g), axis=-1) / np.float32(6)).astype(np.float64))
        s = e4m3_table()[s8].astype(np.float32)[..., None]
        z = np.where(s > 0, g / np.where(s > 0, s, np.float32(1)), np.float32(0)).astype(np.float64)
    a = np.minimum(np.where(np.isnan(z), 0.0, np.abs(z)), 6.0)
    hi = np.clip(np.searchsorted(E2M1, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - E2M1[lo], E2M1[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = (code | (np.signbit(z).astype(np.uint8) << 3)).reshape(*y.shape[:-1], 256, 2)
    return np.concatenate([code[..., 0] | (code[..., 1] << 4), s8], axis=-1)


def widen_cache(pages) -> np.ndarray:
    """Cached rows of any format in fp64, without the tensor scale."""
    if tuple(pages.shape)[-1] == FP4_ROW:
        return widen_fp4(pages)
    return widen_bf16(pages) if "bfloat16" in str(pages.dtype) else widen_e4m3(pages)


def decode_paged_any(q, k_pages, v_pages, page_table, kv_lens, selected=None, *, scale=None, window: int = 0,
                     k_scale: float = 1.0, v_scale: float = 1.0):
    """``(out, lse, weight)`` as decode_paged_tree, of the last q_len tokens of each sequence over a cache of any
    format; with ``selected`` [batch, n_kv_heads, n] over the listed pages alone."""
    qf, pt, kl = widen_bf16(q), _i32(page_table), _i32(kv_lens)
    sel = None if selected is None else _i32(selected)
    bsz, qlen, hq, d = qf.shape
    psz, hk = (int(x) for x in tuple(k_pages.shape)[1:3])
    G = hq // hk
    scale = d ** -0.5 if scale is None else float(scale)
    out, weight = np.zeros(qf.shape), np.zeros(qf.shape)
    lse = np.full((bsz, qlen, hq), -np.inf)
    for b in range(bsz):
        n = int(kl[b])
        here = n - qlen + np.arange(qlen)
        for h in range(hk):
            pages = np.arange(pages_of(n, psz)) if sel is None else sel[b, h][sel[b, h] >= 0]
            j = (pages[:, None] * psz + np.arange(psz)).reshape(-1)
            j = j[j < n]
            vis = j[None] <= here[:, None]
            if window > 0:
                vis &= j[None] > here[:, None] - window
            j, vis = j[vis.any(axis=0)], vis[:, vis.any(axis=0)]
            if not len(j):
                continue
            k = widen_cache(k_pages[pt[b, j // psz], j % psz, h]) * k_scale
            v = widen_cache(v_pages[pt[b, j // psz], j % psz, h]) * v_scale
            for i in range(h * G, (h + 1) * G):
                s = np.where(vis, qf[b, :, i] @ k.T * scale, -np.inf)
                m = s.max(axis=1)
                some = m > -np.inf
                p = np.exp(s - np.where(some, m, 0.0)[:, None])
                l = np.where(some, p.sum(axis=1), 1.0)
                out[b, :, i] = (p @ v) / l[:, None]
                weight[b, :, i] = (p @ np.abs(v)) / l[:, None]
                lse[b, :, i] = np.where(some, m + np.log(l), -np.inf)
    return out, lse, weight


def page_bounds(k_pages, page_table, kv_lens, bounds, q_len: int, q_lens=None) -> np.ndarray:
    """The bounds (fp64 [num_pages, n_kv_heads, 2, 512]) after the call, from ``bounds`` before it."""
    pt, kl = _i32(page_table), _i32(kv_lens)
    psz = int(tuple(k_pages.shape)[1])
    out = widen_bf16(bounds)
    for b in range(len(kl)):
        cnt = q_len if q_lens is None else int(_i32(q_lens)[b])
        n = int(kl[b])
        if cnt == 0:
            continue
        for p in range((n - cnt) // psz, (n - 1) // psz + 1):
            k = widen_cache(k_pages[pt[b, p], :min(psz, n - p * psz)])
            out[pt[b, p], :, 0], out[pt[b, p], :, 1] = k.min(axis=0), k.max(axis=0)
    return out


def page_scores(q, bounds, page_table, kv_lens, b: int, psz: int, kind=np.float64) -> np.ndarray:
    """[n_kv_heads, pages] scores of sequence b: in fp64, or in fp32 in the operation's order of sums."""
    qf, bf = widen_bf16(q).astype(kind), widen_bf16(bounds).astype(kind)
    pt, n = _i32(page_table), int(_i32(kv_lens)[b])
    _, qlen, hq, d = qf.shape
    hk = bf.shape[1]
    w = bf[pt[b, :pages_of(n, psz)]]
    got = np.full((hk, w.shape[0]), -np.inf)
    for h in range(hk):
        for t in range(max(0, qlen - n), qlen):
            for i in range(h * (hq // hk), (h + 1) * (hq // hk)):
                x = np.maximum(qf[b, t, i] * w[:, h, 0], qf[b, t, i] * w[:, h, 1])
                x = x.reshape(-1, 2, 32, 8).transpose(0, 1, 3, 2).reshape(-1, d)
                while x.shape[1] > 1:
                    x = x[:, :x.shape[1] // 2] + x[:, x.shape[1] // 2:]
                got[h] = np.maximum(got[h], x[:, 0])
    return got


def select_pages(q, bounds, page_table, kv_lens, psz: int, n_select: int, n_first: int, n_last: int) -> np.ndarray:
    """[batch, n_kv_heads, n_select] int32."""
    kl = _i32(kv_lens)
    hk = int(tuple(bounds.shape)[1])
    got = np.full((len(kl), hk, n_select), -1, dtype=np.int32)
    for b in range(len(kl)):
        held = pages_of(int(kl[b]), psz)
        if not held:
            continue
        score = page_scores(q, bounds, page_table, kl, b, psz, np.float32)
        # those always chosen, then those with a bound that is not finite, then by the score
        rank = np.full(score.shape, 2)
        rank[~np.isfinite(widen_bf16(bounds)[_i32(page_table)[b, :held]]).all(axis=(2, 3)).T] = 1
        rank[:, :n_first] = 0
        rank[:, max(0, held - n_last):] = 0
        for h in range(hk):
            best = np.sort(np.lexsort((np.where(rank[h] == 2, -score[h], 0.0), rank[h]))[:n_select])
            got[b, h, :len(best)] = best
    return got
