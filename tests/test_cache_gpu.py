"""fa512_cache_append, _compact, _fork and _resize (CUDA) against the plain
references: moved rows, tables and counts exactly, E4M3 codes exactly (the
quotient's rounding to fp32 is part of the operation), and a run of all calls
together as a speculative decoding loop makes them."""
import numpy as np
import pytest
import torch

from head_dim_flashattention_gb300 import workloads
from oracle import paged

pytestmark = pytest.mark.gpu
D = 512


@pytest.fixture(scope="module")
def fa(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    import head_dim_flashattention_gb300 as fa
    fa.load_library()
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def bits(t):
    t = t.cpu()
    return t.numpy() if t.dtype == torch.uint8 else t.view(torch.int16).numpy().view(np.uint16)


def random_pages(shape, fp8, seed):
    g = torch.Generator().manual_seed(seed)
    if fp8:
        return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
    return torch.randint(-32768, 32767, shape, generator=g, dtype=torch.int16).view(torch.bfloat16)


def tables(lens, psz, width, pool, seed, spare_entry):
    """(table [batch, width], counts): a seeded permutation of the pool's pages."""
    perm = np.random.RandomState(seed).permutation(pool)
    t = np.full((len(lens), width), spare_entry, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = paged.pages_of(n, psz)
        t[b, :k] = perm[at:at + k]
        at += k
    refs = np.zeros(pool, dtype=np.int32)
    refs[perm[:at]] = 1
    return torch.from_numpy(t), torch.from_numpy(refs)


FP8 = pytest.mark.parametrize("fp8", [False, True])


# ---------------------------------------------------------------------- append

@FP8
@pytest.mark.parametrize("q_len,psz,hk", [(1, 64, 4), (1, 16, 1), (7, 32, 3), (130, 64, 4), (300, 256, 2)])
def test_append(fa, q_len, psz, hk, fp8):
    lens = [q_len, q_len + 77, 2 * q_len + 5]
    width = paged.pages_of(max(lens), psz) + 1
    pool = 3 * width + 2
    pt, _ = tables(lens, psz, width, pool, 91, 10 ** 7)
    k, v = random_pages((pool, psz, hk, D), fp8, 1), random_pages((pool, psz, hk, D), fp8, 2)
    kn = workloads.randn_bf16((3, q_len, hk, D), 93)
    vn = workloads.randn_bf16((3, q_len, hk, D), 94) * 100
    for ql in (None, i32([q_len, 0, max(0, q_len - 1)])):
        kc, vc = k.cuda(), v.cuda()
        args = (kn.cuda(), vn.cuda(), kc, vc, pt.cuda(), i32(lens).cuda())
        kw = {"q_lens": None if ql is None else ql.cuda()}
        ks, vs = (0.013, 0.11) if fp8 else (None, None)
        if fp8:
            fa.fa512_cache_append_fp8(*args, k_scale=ks, v_scale=vs, **kw)
        else:
            fa.fa512_cache_append(*args, **kw)
        assert fa.fa512_device_status() == 0
        assert np.array_equal(bits(kc), paged.cache_append(kn, bits(k), pt, lens, ql, ks))
        assert np.array_equal(bits(vc), paged.cache_append(vn, bits(v), pt, lens, ql, vs))


@FP8
def test_append_takes_slices_of_a_fused_projection(fa, fp8):
    lens, hq, hk, psz = [70, 33], 8, 4, 32
    pt, _ = tables(lens, psz, 3, 8, 95, -1)
    qkv = workloads.randn_bf16((2, 5, hq + 2 * hk, D), 96).cuda()
    kn, vn = qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
    k, v = random_pages((8, psz, hk, D), fp8, 3), random_pages((8, psz, hk, D), fp8, 4)
    kc, vc = k.cuda(), v.cuda()
    f = fa.fa512_cache_append_fp8 if fp8 else fa.fa512_cache_append
    f(kn, vn, kc, vc, pt.cuda(), i32(lens).cuda())
    s = 1.0 if fp8 else None
    assert np.array_equal(bits(kc), paged.cache_append(kn.cpu().contiguous(), bits(k), pt, lens, None, s))
    assert np.array_equal(bits(vc), paged.cache_append(vn.cpu().contiguous(), bits(v), pt, lens, None, s))
    # a token stride of 0 (one token's rows for every token) is a stride like others
    one = qkv[:, :1, :hk].expand(2, 5, hk, D)
    f(one, one, kc, vc, pt.cuda(), i32(lens).cuda())
    assert np.array_equal(bits(kc), paged.cache_append(one.cpu().contiguous(), bits(k), pt, lens, None, s))


def test_append_rounds_every_bf16_to_the_nearest_code(fa):
    """All 65,536 bf16 values (infinities and NaN among them) under a power of two and another scale."""
    every = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    kn = every.view(1, 32, 4, D)
    pt = i32([[0]])
    for scale in (1.0, 1 / 32, 0.013, 3.0, 2.0 ** -126, 2.0 ** 127):
        k = torch.zeros((1, 32, 4, D), dtype=torch.uint8, device="cuda")
        v = torch.zeros_like(k)
        fa.fa512_cache_append_fp8(kn.cuda(), kn.cuda(), k, v, pt.cuda(), i32([32]).cuda(), k_scale=scale,
                                  v_scale=scale)
        want = paged.cache_append(kn, np.zeros((1, 32, 4, D), np.uint8), pt, [32], None, scale)
        got, ref = bits(k), want
        # codes of NaN differ in their sign at most
        nan = (ref & 0x7F) == 0x7F
        assert np.array_equal(got[~nan], ref[~nan]), scale
        assert np.all((got[nan] & 0x7F) == 0x7F)
        assert np.array_equal(bits(v), got)


def test_append_reports_what_it_cannot_place(fa):
    psz, hk = 16, 2
    pages = random_pages((4, psz, hk, D), False, 5)
    before = bits(pages)
    kn = workloads.randn_bf16((1, 3, hk, D), 97).cuda()
    for pt, n, ql in ([[99, 1]], [10], None), ([[-1, 1]], [10], None), ([[0, 1]], [33 + 3], None), ([[0, 1]], [2], None), \
            ([[0, 1]], [10], [-2]):
        k = pages.cuda()
        fa.fa512_cache_append(kn, kn, k, k.clone(), i32(pt).cuda(), i32(n).cuda(),
                              q_lens=None if ql is None else i32(ql).cuda())
        assert fa.fa512_device_status() == 6
        want = before.copy()
        if n == [2]:   # a length of 2 with 3 new tokens: the two that have a place are written
            want[0, :2] = bits(kn)[0, 1:]
        assert np.array_equal(bits(k), want), (pt, n, ql)


# --------------------------------------------------------------------- compact

@FP8
@pytest.mark.parametrize("layers,hk,psz,nodes,most", [(1, 4, 64, 8, 8), (3, 1, 16, 40, 20), (2, 3, 32, 64, 1),
                                                      (1, 2, 256, 300, 300)])
def test_compact(fa, layers, hk, psz, nodes, most, fp8):
    rng = np.random.RandomState(nodes)
    lens = [nodes, nodes + 1, nodes + 111, 2 * nodes + 15, nodes]
    cnts = [nodes, nodes // 2, nodes, max(1, nodes - 3), 0]
    width = paged.pages_of(max(lens), psz)
    pool = 5 * width + 1
    pt, _ = tables(lens, psz, width, pool, 98, 10 ** 7)
    acc, na = np.full((5, most), -7, dtype=np.int32), np.zeros(5, dtype=np.int32)
    for b, c in enumerate(cnts):
        na[b] = min(c, most) if b % 2 == 0 else rng.randint(0, min(c, most) + 1)
        acc[b, :na[b]] = np.sort(rng.permutation(c)[:na[b]])
    k, v = random_pages((layers, pool, psz, hk, D), fp8, 6), random_pages((layers, pool, psz, hk, D), fp8, 7)
    for ql in (i32(cnts), None) if all(a < nodes for a in acc.max(1)) else (i32(cnts),):
        if ql is None and min(lens) < nodes:
            continue
        kc, vc = k.cuda(), v.cuda()
        new = fa.fa512_cache_compact(kc, vc, pt.cuda(), i32(lens).cuda(), torch.from_numpy(acc).cuda(),
                                     torch.from_numpy(na).cuda(), q_len=nodes, q_lens=None if ql is None else ql.cuda())
        assert fa.fa512_device_status() == 0
        want, n = paged.cache_compact(bits(k), pt, lens, acc, na, nodes, ql)
        assert np.array_equal(new.cpu().numpy(), n)
        assert np.array_equal(bits(kc), want)
        assert np.array_equal(bits(vc), paged.cache_compact(bits(v), pt, lens, acc, na, nodes, ql)[0])


def test_compact_takes_one_layer_without_its_dimension(fa):
    k = random_pages((3, 16, 2, D), False, 8)
    pt, lens = i32([[2, 0]]), [20]
    kc = k.cuda()
    new = fa.fa512_cache_compact(kc, kc.clone(), pt.cuda(), i32(lens).cuda(), i32([[1, 5]]).cuda(), i32([2]).cuda(),
                                 q_len=6)
    want, n = paged.cache_compact(bits(k)[None], pt, lens, [[1, 5]], [2], 6)
    assert np.array_equal(bits(kc), want[0]) and new.tolist() == n.tolist()


def test_compact_leaves_a_sequence_that_makes_no_sense(fa):
    """Not rising, outside the tree, too many, impossible lengths: recorded, nothing moved, the length kept;
    the other sequences are done."""
    pt = i32([[0, 1], [2, 3]])
    good = ([0, 2, 3], 3)
    for acc, na, n, cnt in (([0, 2, 2], 3, 20, 8), ([3, 1, 4], 3, 20, 8), ([0, 1, 8], 3, 20, 8), ([-1, 1, 2], 3, 20, 8),
                            ([0, 1, 2], 4, 20, 8), ([0, 1, 2], -1, 20, 8), ([0, 1, 2], 3, 4, 8), ([0, 1, 2], 3, 40, 8),
                            ([0, 1, 2], 3, 20, 9), ([0, 1, 2], 3, 20, 2), ([0, 1, 2], 3, 20, -1)):
        k = random_pages((1, 4, 16, 1, D), False, 9)
        kc, vc = k.cuda(), k.cuda()
        new = fa.fa512_cache_compact(kc, vc, pt.cuda(), i32([n, 30]).cuda(), i32([acc, good[0]]).cuda(),
                                     i32([na, good[1]]).cuda(), q_len=8, q_lens=i32([cnt, 8]).cuda())
        assert fa.fa512_device_status() == 6, (acc, na, n, cnt)
        want, _ = paged.cache_compact(bits(k), i32([[2, 3]]), [30], [good[0]], [3], 8)
        assert np.array_equal(bits(kc), want) and np.array_equal(bits(vc), want)
        assert new.tolist() == [n, 25]
    # a page outside the pool: its rows are left out
    k = random_pages((1, 4, 16, 1, D), False, 10)
    kc = k.cuda()
    fa.fa512_cache_compact(kc, kc.clone(), i32([[0, 77], [2, 3]]).cuda(), i32([20, 30]).cuda(),
                           i32([[1, 7, -1], [0, 2, 3]]).cuda(), i32([2, 3]).cuda(), q_len=8)
    assert fa.fa512_device_status() == 6
    want, _ = paged.cache_compact(bits(k), i32([[0, 0], [2, 3]]), [20, 30], [[1, -1, -1], [0, 2, 3]], [1, 3], 8)
    assert np.array_equal(bits(kc), want)


# ------------------------------------------------------------- fork and resize

@FP8
@pytest.mark.parametrize("layers,hk,psz,lens,parents", [
    (1, 4, 64, [130, 64, 1], [0, 0, 0, 2, 1, 1]),
    (2, 1, 16, [16, 32, 48], [2, 2, 0, 1]),                       # whole pages only: nothing to copy
    (3, 2, 32, [31, 33, 0, 95], [3, 3, 2, 2, 0, 3, 0]),           # an empty sequence, one without children
    (1, 1, 256, [700, 255], [1] * 40),
    (2, 3, 16, [5], [0]),
    (1, 1, 16, [9, 300, 17], [])])                                # everybody ends
def test_fork(fa, layers, hk, psz, lens, parents, fp8):
    width = paged.pages_of(max(lens), psz) + 2
    pool = sum(paged.pages_of(n, psz) for n in lens) + len(parents) + 3
    pt, refs = tables(lens, psz, width, pool, 99, 10 ** 7)
    refs[-1] += 5                                                  # another holder's page
    k, v = random_pages((layers, pool, psz, hk, D), fp8, 11), random_pages((layers, pool, psz, hk, D), fp8, 12)
    wk, wv, wt, wl, wr = paged.cache_fork(bits(k), bits(v), pt, lens, np.array(parents, dtype=np.int32), refs)
    for in_place in (False, True):
        kc, vc, rc = k.cuda(), v.cuda(), refs.cuda()
        t, n, r = fa.fa512_cache_fork(kc, vc, pt.cuda(), i32(lens).cuda(), i32(parents).cuda(), rc,
                                      new_page_refs=rc if in_place else None)
        assert fa.fa512_device_status() == 0
        assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(n.cpu().numpy(), wl)
        assert np.array_equal(r.cpu().numpy(), wr)
        assert np.array_equal(bits(kc), wk) and np.array_equal(bits(vc), wv)
        assert in_place or torch.equal(rc.cpu(), refs)


def test_fork_without_room_and_with_bad_entries(fa):
    psz = 16
    k = random_pages((1, 4, psz, 1, D), False, 13)
    pt, refs = i32([[3, 1], [0, -1]]), i32([1, 1, 0, 1])
    kc = k.cuda()
    t, n, r = fa.fa512_cache_fork(kc, kc.clone(), pt.cuda(), i32([20, 3]).cuda(), i32([0, 0, 0, 1]).cuda(), refs.cuda())
    assert fa.fa512_device_status() == 7                           # FA512_ERR_OUT_OF_PAGES
    assert t.tolist() == [[3, 1], [3, 2], [3, -1], [0, -1]] and r.tolist() == [1, 1, 1, 3] and n.tolist() == [20] * 3 + [3]
    assert np.array_equal(bits(kc)[0, 2, :4], bits(k)[0, 1, :4])
    assert np.array_equal(bits(kc)[0, 2, 4:], bits(k)[0, 2, 4:])   # rows behind the length are not touched
    for parents, lens, table in (([0, 7], [20, 3], pt), ([0, -1], [20, 3], pt), ([0, 1], [33, 3], pt),
                                 ([0, 1], [-4, 3], pt), ([0, 1], [20, 3], i32([[3, 9], [0, -1]]))):
        kc = k.cuda()
        fa.fa512_cache_fork(kc, kc.clone(), table.cuda(), i32(lens).cuda(), i32(parents).cuda(), refs.cuda())
        assert fa.fa512_device_status() == 6


@pytest.mark.parametrize("psz,batch,top,spare", [(64, 1, 100, 3), (16, 40, 500, 900), (32, 1500, 90, 4000),
                                                 (256, 7, 3000, 5), (64, 3, 64, 30000)])
def test_resize(fa, psz, batch, top, spare):
    rng = np.random.RandomState(batch)
    old = rng.randint(0, top + 1, batch)
    new = rng.randint(0, top + 1, batch)
    width = paged.pages_of(top, psz) + 1
    pool = sum(paged.pages_of(int(n), psz) for n in old) + spare
    need = sum(max(0, paged.pages_of(int(a), psz) - paged.pages_of(int(b), psz)) for a, b in zip(new, old))
    free = spare + sum(max(0, paged.pages_of(int(b), psz) - paged.pages_of(int(a), psz)) for a, b in zip(new, old))
    pt, refs = tables(list(old), psz, width, pool, 100, 10 ** 7)
    wt, wr = paged.cache_resize(pt, old, new, refs, psz)
    for in_place in (False, True):
        tc, rc = pt.cuda(), refs.cuda()
        t, r = fa.fa512_cache_resize(tc, i32(list(old)).cuda(), i32(list(new)).cuda(), rc, tc if in_place else None,
                                     rc if in_place else None, page_size=psz)
        assert fa.fa512_device_status() == (7 if need > free else 0)
        assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(r.cpu().numpy(), wr)


def test_resize_of_nothing_and_bad_entries(fa):
    refs = i32([0, 2, 0]).cuda()
    t, r = fa.fa512_cache_resize(torch.empty((0, 2), dtype=torch.int32, device="cuda"), i32([]).cuda(), i32([]).cuda(),
                                 refs, page_size=64)
    assert t.shape == (0, 2) and torch.equal(r, refs) and fa.fa512_device_status() == 0
    for pt, a, z in ([[5, 1]], [128], [64]), ([[1, 0]], [129], [64]), ([[1, 0]], [64], [1000]):
        fa.fa512_cache_resize(i32(pt).cuda(), i32(a).cuda(), i32(z).cuda(), refs, page_size=64)
        assert fa.fa512_device_status() == 6


# -------------------------------------------------------------- all together

@FP8
def test_a_speculative_decoding_loop(fa, fp8):
    """Prompts are appended, forked into samples, and three steps draft a tree each: resize, append, tree attention,
    compact, resize.  After every step the attention over the cache agrees with the reference over the tokens that
    the sequences hold, kept beside on the CPU, and the counts with the tables."""
    hq, hk, psz, pool, nodes, scale = 8, 4, 16, 200, 11, (1 / 32 if fp8 else None)
    rng = np.random.RandomState(5)
    dt = torch.uint8 if fp8 else torch.bfloat16
    k = torch.zeros((pool, psz, hk, D), dtype=dt, device="cuda")
    v = torch.zeros_like(k)
    kw = {"k_scale": scale, "v_scale": scale} if fp8 else {}
    append = fa.fa512_cache_append_fp8 if fp8 else fa.fa512_cache_append
    attend = fa.fa512_decode_paged_tree_fp8 if fp8 else fa.fa512_decode_paged_tree

    def new_rows(b, t, seed):
        return workloads.randn_bf16((b, t, hk, D), seed), workloads.randn_bf16((b, t, hk, D), seed + 1)

    width = 12
    zero = i32([0, 0]).cuda()
    lens = i32([75, 48]).cuda()
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table, refs = fa.fa512_cache_resize(table, zero, lens, refs, page_size=psz)
    kn, vn = new_rows(2, 75, 500)
    append(kn.cuda(), vn.cuda(), k, v, table, lens, q_lens=lens, **kw)
    held = [(kn[b, :n], vn[b, :n]) for b, n in enumerate([75, 48])]
    parents = [0, 1, 0, 1, 1]
    table, lens, refs = fa.fa512_cache_fork(k, v, table, lens, i32(parents).cuda(), refs)
    held = [held[a] for a in parents]
    for step in range(3):
        b = len(held)
        grown = lens + nodes
        table, refs = fa.fa512_cache_resize(table, lens, grown, refs, page_size=psz)
        kn, vn = new_rows(b, nodes, 600 + 10 * step)
        append(kn.cuda(), vn.cuda(), k, v, table, grown, **kw)
        words = np.zeros((b, nodes, 1), dtype=np.int64)
        up = np.array([[rng.randint(-1, i) if i else -1 for i in range(nodes)] for _ in range(b)])
        for s in range(b):
            for i in range(nodes):
                words[s, i, 0] = (words[s, up[s, i], 0] if up[s, i] >= 0 else 0) | 1 << i
        mask = torch.from_numpy(words.astype(np.int32))
        q = workloads.randn_bf16((b, nodes, hq, D), 700 + step)
        out, lse = attend(q.cuda(), k, v, table, grown, mask.cuda(), **kw)
        # the reference, over the tokens themselves laid out one page after another
        cap = max(len(x[0]) for x in held) + nodes
        lin = [torch.zeros((b, cap, hk, D), dtype=torch.bfloat16) for _ in range(2)]
        for s, (a, c) in enumerate(held):
            for x, have, new in ((lin[0], a, kn), (lin[1], c, vn)):
                x[s, :len(have)], x[s, len(have):len(have) + nodes] = have, new[s]
        if fp8:
            lin = [torch.from_numpy(paged.e4m3_round(paged.widen_bf16(x) / scale)) for x in lin]
        want = paged.decode_paged_tree(q, lin[0], lin[1], torch.arange(b, dtype=torch.int32)[:, None], grown.cpu(), mask, **kw)
        ro, rl, weight = want
        err = np.abs(out.float().cpu().numpy() - ro)
        assert np.all(err <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 1e-3) * weight + 1e-6)
        assert np.max(np.abs(lse.cpu().numpy() - rl)) <= 1e-3
        # accept a path of each tree
        acc, na = np.full((b, nodes), -1, dtype=np.int32), np.zeros(b, dtype=np.int32)
        for s in range(b):
            path, i = [], rng.randint(nodes)
            while i >= 0:
                path.append(i)
                i = up[s, i]
            path = path[::-1]
            acc[s, :len(path)], na[s] = path, len(path)
            held[s] = (torch.cat([held[s][0], kn[s, path]]), torch.cat([held[s][1], vn[s, path]]))
        lens = fa.fa512_cache_compact(k, v, table, grown, torch.from_numpy(acc).cuda(), torch.from_numpy(na).cuda(), q_len=nodes)
        table, refs = fa.fa512_cache_resize(table, grown, lens, refs, page_size=psz)
        assert lens.tolist() == [len(x[0]) for x in held]
        t = table.cpu().numpy()
        assert np.array_equal(refs.cpu().numpy(), np.bincount(t[t >= 0], minlength=pool))
        if step == 1:
            parents = [3, 3, 0, 4]
            table, lens, refs = fa.fa512_cache_fork(k, v, table, lens, i32(parents).cuda(), refs)
            held = [held[a] for a in parents]
    assert fa.fa512_device_status() == 0


def test_the_page_calls_can_be_captured(fa):
    """Resize and fork in one graph, replayed on new lengths and parents."""
    psz, pool = 16, 60
    pt, refs = tables([40, 33, 7], psz, 8, pool, 101, -1)
    k = random_pages((1, pool, psz, 1, D), False, 14)
    kc, vc, tc, rc = k.cuda(), k.cuda(), pt.cuda(), refs.cuda()
    a, z, par = i32([40, 33, 7]).cuda(), i32([60, 10, 7]).cuda(), i32([0, 0, 1]).cuda()

    def run():
        t, r = fa.fa512_cache_resize(tc, a, z, rc, page_size=psz)
        return (t, r) + fa.fa512_cache_fork(kc, vc, t, z, par, r)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for new, parents in (([60, 10, 7], [0, 0, 1]), ([0, 100, 20], [1, 2, 1]), ([17, 33, 128], [2, 2, 2])):
        z.copy_(i32(new))
        par.copy_(i32(parents))
        kc.copy_(k)
        g.replay()
        torch.cuda.synchronize()
        t, r = paged.cache_resize(pt, [40, 33, 7], new, refs, psz)
        wk, _, wt, wl, wr = paged.cache_fork(bits(k), bits(k), t, new, np.array(parents, dtype=np.int32), r)
        for got, want in zip(out, (t, r, wt, wl, wr)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert np.array_equal(bits(kc), wk)
    assert fa.fa512_device_status() == 0


@FP8
def test_rows_far_into_a_large_pool(fa, fp8):
    """Append, compact and fork past 32 bits of elements give what they give in a small pool."""
    psz, hk, n = 64, 4, 24
    far = 34000 if fp8 else 17000
    dt = torch.uint8 if fp8 else torch.bfloat16
    append = fa.fa512_cache_append_fp8 if fp8 else fa.fa512_cache_append
    kw = {"k_scale": 0.03, "v_scale": 0.5} if fp8 else {}
    pt, refs = tables([300, 170], psz, 8, n, 110, -1)
    rows = [workloads.randn_bf16((2, 300, hk, D), 520 + i).cuda() for i in range(2)]
    acc = torch.tensor([[0, 3, 4, 9], [2, 5, 6, 7]], dtype=torch.int32).cuda()
    tails = []
    for first in (0, far):
        k, v = (torch.empty((1, first + n, psz, hk, D), dtype=dt, device="cuda") for _ in range(2))
        k[:, first:].zero_()
        v[:, first:].zero_()
        table = torch.where(pt >= 0, pt + first, pt).cuda()
        counts = torch.cat([torch.ones(first, dtype=torch.int32), refs]).cuda()
        lens = i32([300, 170]).cuda()
        append(rows[0], rows[1], k[0], v[0], table, lens, q_lens=lens, **kw)
        lens = fa.fa512_cache_compact(k, v, table, lens, acc, i32([4, 3]).cuda(), q_len=10)
        table, lens, counts = fa.fa512_cache_fork(k, v, table, lens, i32([0, 1, 0, 0]).cuda(), counts)
        table = table.cpu()
        tails.append((bits(k[:, first:]), bits(v[:, first:]), torch.where(table >= 0, table - first, table), lens.cpu(),
                      counts[first:].cpu()))
        del k, v
    for a, b in zip(*tails):
        assert np.array_equal(np.asarray(a), np.asarray(b))
    assert np.any(tails[0][0] != 0) and fa.fa512_device_status() == 0


def test_the_last_page_and_a_full_pool_on_two_streams(fa):
    """Resizes of two caches at once; one takes its pool's last free page, the other one more than there is."""
    psz, pool = 16, 40
    jobs = []
    for new in ([320, 320], [320, 336]):
        table = torch.full((2, 30), -1, dtype=torch.int32, device="cuda")
        jobs.append((table, i32([0, 0]).cuda(), i32(new).cuda(), torch.zeros(pool, dtype=torch.int32, device="cuda"),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [fa.fa512_cache_resize(t, z, n, r, page_size=psz, stream=st) for t, z, n, r, st in jobs]
    torch.cuda.synchronize()
    assert fa.fa512_device_status() == 7 and fa.fa512_device_status() == 0
    for t, r in outs:
        t = t.cpu().numpy()
        assert sorted(t[t >= 0]) == list(range(pool)) and np.all(r.cpu().numpy() == 1)


def test_page_plans_of_large_caches(fa):
    """As many blocks as the plan takes: hundreds of sequences of hundreds of pages, a pool of tens of thousands."""
    test_resize(fa, 16, 512, 3200, 3001)
    psz, pool = 16, 70001
    rng = np.random.RandomState(7)
    lens = rng.randint(0, 1700, 500)
    parents = rng.randint(0, 500, 700).astype(np.int32)
    pt, refs = tables(list(lens), psz, 110, pool, 111, 10 ** 7)
    none = np.zeros((0, pool, psz, 1, D), dtype=np.uint16)
    _, _, wt, wl, wr = paged.cache_fork(none, none, pt, lens, parents, refs)
    k = torch.empty((0, pool, psz, 1, D), dtype=torch.bfloat16, device="cuda")
    t, n, r = fa.fa512_cache_fork(k, k, pt.cuda(), i32(list(lens)).cuda(), torch.from_numpy(parents).cuda(), refs.cuda())
    assert fa.fa512_device_status() == 0
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(n.cpu().numpy(), wl)
    assert np.array_equal(r.cpu().numpy(), wr)
