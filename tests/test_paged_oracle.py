"""CPU pins of the drafted-token and cache references, and the refusals of the
calls they check: everything here answers without a device."""
import numpy as np
import pytest
import torch

import __graft_entry__
import head_dim_flashattention_gb300 as fa
import oracle
from head_dim_flashattention_gb300 import workloads
from oracle import paged


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return fa.load_library()


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("window", [0, 1, 20])
def test_without_a_mask_the_tree_is_the_causal_run(window):
    pc = workloads.paged_decode_inputs(3, [2, 129, 300], 8, 4, 64, seed=61)
    q = workloads.draft_queries(3, 4, 8, seed=61)
    o, l, _ = paged.decode_paged_tree(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, window=window)
    ro, rl = oracle.decode_paged_q(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, window=window)
    np.testing.assert_allclose(o, ro, atol=1e-12)
    np.testing.assert_allclose(l, rl, atol=1e-12)


def test_a_lower_triangle_mask_is_the_causal_run_and_depth_is_position():
    pc = workloads.paged_decode_inputs(2, [90, 200], 4, 4, 16, seed=62)
    q = workloads.draft_queries(2, 40, 4, seed=62)
    words = torch.zeros((2, 40, 2), dtype=torch.int64)
    for t in range(40):
        for c in range(t + 1):
            words[:, t, c // 32] |= 1 << (c % 32)
    mask = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    a = paged.decode_paged_tree(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, mask, window=30, n_sinks=5)
    b = paged.decode_paged_tree(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, None, window=30, n_sinks=5)
    np.testing.assert_array_equal(a[0], b[0])
    np.testing.assert_array_equal(a[1], b[1])


def test_sinks_add_exactly_the_first_positions():
    vis = paged.tree_visible(None, 0, 100, 3, window=10, n_sinks=4)
    assert np.nonzero(vis[0])[0].tolist() == list(range(4)) + list(range(88, 98))
    assert np.nonzero(vis[2])[0].tolist() == list(range(4)) + list(range(90, 100))
    # siblings sit at the same place: neither pushes a key out of the other's window
    mask = torch.tensor([[[1], [2], [5]]], dtype=torch.int32)
    vis = paged.tree_visible(mask, 0, 100, 3, window=10, n_sinks=0)
    assert np.nonzero(vis[0])[0].tolist() == list(range(88, 98))
    assert np.nonzero(vis[1])[0].tolist() == list(range(88, 97)) + [98]
    assert np.nonzero(vis[2])[0].tolist() == list(range(89, 98)) + [99]


def test_e4m3_rounding_of_every_code_and_midpoint():
    v = oracle.e4m3_table()[:127]
    assert np.array_equal(paged.e4m3_round(v), np.arange(127, dtype=np.uint8))
    mid = (v[1:] + v[:-1]) / 2
    even = np.arange(126) + (np.arange(126) % 2)
    assert np.array_equal(paged.e4m3_round(mid), even.astype(np.uint8))
    assert paged.e4m3_round(np.array([1e9, -np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x7F]


def test_fork_and_resize_keep_every_count():
    """The counts always say how many table entries refer to a page."""
    rng = np.random.RandomState(3)
    psz, pool = 16, 40
    lens = np.array([30, 16, 47, 5], dtype=np.int32)
    table = np.full((4, 6), -1, dtype=np.int32)
    perm, at = rng.permutation(pool), 0
    for b, n in enumerate(lens):
        for i in range(paged.pages_of(int(n), psz)):
            table[b, i] = perm[at]
            at += 1
    refs = np.bincount(table[table >= 0], minlength=pool).astype(np.int32)
    k = rng.randint(0, 255, (1, pool, psz, 1, 4)).astype(np.uint8)
    k2, v2, t2, l2, r2 = paged.cache_fork(k, k, table, lens, np.array([2, 0, 2, 2, 1], dtype=np.int32), refs)
    assert np.array_equal(r2, np.bincount(t2[t2 >= 0], minlength=pool))
    for c, a in enumerate([2, 0, 2, 2, 1]):
        for pos in range(int(lens[a])):
            assert np.array_equal(k2[0, t2[c, pos // psz], pos % psz], k[0, table[a, pos // psz], pos % psz])
    t3, r3 = paged.cache_resize(t2, l2, np.array([47, 96, 0, 20, 17], dtype=np.int32), r2, psz)
    assert np.array_equal(r3, np.bincount(t3[t3 >= 0], minlength=pool))


# ------------------------------------------------------- refusals before a launch

def _tree(lib, fp8=False, **kw):
    a = dict(q=16, kp=16, vp=16, pt=16, kl=16, ql=None, mask=None, out=16, lse=None, b=2, qlen=4, hq=8, hk=4,
             ps=64, npages=10, mpps=4, maxlen=200, scale=0.05, ks=0.1, vs=0.1, window=0, sinks=0, splits=2,
             ws=256, wsb=1 << 30)
    assert set(kw) <= set(a)
    a.update(kw)
    f = lib.fa512_decode_paged_tree_fp8 if fp8 else lib.fa512_decode_paged_tree
    scales = (a["scale"], a["ks"], a["vs"]) if fp8 else (a["scale"],)
    return f(a["q"], a["kp"], a["vp"], a["pt"], a["kl"], a["ql"], a["mask"], a["out"], a["lse"], a["b"],
             a["qlen"], a["hq"], a["hk"], a["ps"], a["npages"], a["mpps"], a["maxlen"], *scales, a["window"],
             a["sinks"], a["splits"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_refusals(lib, fp8):
    inf, nan = float("inf"), float("nan")
    for want, kw in [(1, dict(b=-1)), (1, dict(qlen=0)), (1, dict(hq=6)), (1, dict(hk=0)), (1, dict(npages=0)),
                     (1, dict(mpps=0)), (1, dict(maxlen=300)), (1, dict(maxlen=-1)), (1, dict(splits=-1)),
                     (1, dict(splits=2000)), (1, dict(sinks=-1)), (1, dict(scale=nan)), (1, dict(scale=inf)),
                     (1, dict(q=None)), (1, dict(pt=None)), (1, dict(kl=None)), (1, dict(out=None)),
                     (1, dict(q=8)), (1, dict(kp=24)), (1, dict(out=40)), (1, dict(mask=18)), (1, dict(ql=17)),
                     (1, dict(lse=2)), (2, dict(hq=516, hk=4)), (2, dict(ps=48)), (2, dict(mask=16, qlen=257)),
                     (2, dict(npages=1 << 24, ps=256)), (2, dict(b=65536)), (2, dict(b=65535, qlen=2)),
                     (5, dict(ws=None)), (5, dict(wsb=1000)), (5, dict(ws=272)), (0, dict(b=0, q=None))]:
        assert _tree(lib, fp8, **kw) == want, kw
    if fp8:
        assert _tree(lib, True, ks=inf) == 1 and _tree(lib, True, vs=nan) == 1


def test_tree_workspace(lib):
    w = fa.fa512_decode_workspace_bytes_tree
    rows = 2 * 9 * 8 * 3
    # the partials, their (m, l) and the segment counts of 2 x 4 items
    assert w(2, 9, 8, 4, 4096, 0, 0, 3) == rows * 2048 + (rows * 8 + 255) // 256 * 256 + 256
    assert w(2, 9, 8, 4, 4096, 0, 0, 1) == 256          # one split: nothing to keep
    assert w(-1, 9, 8, 4, 4096) == 0 and w(2, 0, 8, 4, 4096) == 0 and w(2, 9, 8, 3, 4096) == 0
    assert w(2, 9, 8, 4, 4096, 0, -1) == 0 and w(2, 9, 8, 4, 4096, 0, 0, 2000) == 0
    s = fa.fa512_decode_auto_splits_tree(2, 9, 8, 4, 4096)
    assert 1 <= s <= 33 and w(2, 9, 8, 4, 4096) == w(2, 9, 8, 4, 4096, 0, 0, s)
    assert fa.fa512_decode_auto_splits_tree(1, 1, 8, 4, 0) == 1


def _append(lib, fp8=False, **kw):
    a = dict(kn=16, vn=16, kb=2048, kt=2048, vb=2048, vt=2048, kp=16, vp=16, pt=16, kl=16, ql=None, ks=0.1,
             vs=0.1, b=2, qlen=4, hk=4, ps=64, npages=10, mpps=4)
    assert set(kw) <= set(a)
    a.update(kw)
    f = lib.fa512_cache_append_fp8 if fp8 else lib.fa512_cache_append
    scales = (a["ks"], a["vs"]) if fp8 else ()
    return f(a["kn"], a["vn"], a["kb"], a["kt"], a["vb"], a["vt"], a["kp"], a["vp"], a["pt"], a["kl"], a["ql"],
             *scales, a["b"], a["qlen"], a["hk"], a["ps"], a["npages"], a["mpps"], None)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(lib, fp8):
    for want, kw in [(1, dict(b=-1)), (1, dict(qlen=-1)), (1, dict(hk=0)), (2, dict(ps=8)), (1, dict(npages=0)),
                     (1, dict(kt=2052)), (1, dict(vb=4)), (1, dict(kn=None)), (1, dict(vn=24)), (1, dict(kp=8)),
                     (1, dict(pt=18)), (1, dict(ql=1)), (2, dict(b=65536)), (2, dict(qlen=1 << 28)),
                     (0, dict(b=0, kn=None)), (0, dict(qlen=0, kn=None))]:
        assert _append(lib, fp8, **kw) == want, kw
    if fp8:
        for bad in (0.0, -1.0, float("inf"), float("nan")):
            assert _append(lib, True, ks=bad) == 1 and _append(lib, True, vs=bad) == 1


def _compact(lib, **kw):
    a = dict(k=4096, v=4096, pt=1 << 20, kl=2 << 20, ql=None, acc=3 << 20, na=4 << 20, new=5 << 20, layers=1, b=2,
             qlen=4, most=3, hk=4, eb=2, ps=64, npages=10, mpps=4)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.fa512_cache_compact(a["k"], a["v"], a["pt"], a["kl"], a["ql"], a["acc"], a["na"], a["new"],
                                   a["layers"], a["b"], a["qlen"], a["most"], a["hk"], a["eb"], a["ps"],
                                   a["npages"], a["mpps"], None)


def test_compact_refusals(lib):
    for want, kw in [(1, dict(b=-1)), (1, dict(layers=-1)), (1, dict(qlen=-1)), (1, dict(most=-1)), (1, dict(eb=4)),
                     (1, dict(hk=0)), (2, dict(ps=20)), (1, dict(npages=0)), (2, dict(most=1025)),
                     (1, dict(k=None)), (1, dict(na=None)), (1, dict(acc=None)), (1, dict(new=None)),
                     (1, dict(v=4100)), (1, dict(kl=(2 << 20) + 2)), (1, dict(new=2 << 20)),
                     (1, dict(new=(4 << 20) + 4)), (2, dict(b=65536)), (2, dict(npages=1 << 26)),
                     (0, dict(b=0, k=None))]:
        assert _compact(lib, **kw) == want, kw


def _fork(lib, **kw):
    a = dict(k=4096, v=4096, pt=1 << 20, kl=2 << 20, par=3 << 20, refs=4 << 20, npt=5 << 20, nkl=6 << 20,
             nrefs=7 << 20, layers=1, b=2, kids=3, hk=4, eb=2, ps=64, npages=10, mpps=4)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.fa512_cache_fork(a["k"], a["v"], a["pt"], a["kl"], a["par"], a["refs"], a["npt"], a["nkl"],
                                a["nrefs"], a["layers"], a["b"], a["kids"], a["hk"], a["eb"], a["ps"],
                                a["npages"], a["mpps"], None)


def test_fork_refusals(lib):
    for want, kw in [(1, dict(b=-1)), (1, dict(kids=-1)), (1, dict(layers=-1)), (1, dict(eb=3)), (2, dict(ps=7)),
                     (2, dict(b=8193)), (2, dict(kids=8193)), (1, dict(refs=None)), (1, dict(nrefs=None)),
                     (1, dict(par=None)), (1, dict(npt=None)), (1, dict(k=None)), (1, dict(k=4104)),
                     (1, dict(par=(3 << 20) + 1)), (1, dict(npt=1 << 20)), (1, dict(nkl=2 << 20)),
                     (1, dict(nrefs=(4 << 20) + 4)), (1, dict(nkl=3 << 20))]:
        assert _fork(lib, **kw) == want, kw


def _resize(lib, **kw):
    a = dict(pt=1 << 20, kl=2 << 20, nkl=3 << 20, refs=4 << 20, npt=5 << 20, nrefs=6 << 20, b=2, ps=64, npages=10,
             mpps=4)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.fa512_cache_resize(a["pt"], a["kl"], a["nkl"], a["refs"], a["npt"], a["nrefs"], a["b"], a["ps"],
                                  a["npages"], a["mpps"], None)


def test_resize_refusals(lib):
    for want, kw in [(1, dict(b=-1)), (2, dict(ps=65)), (2, dict(b=8193)), (1, dict(npages=0)), (1, dict(mpps=0)),
                     (1, dict(refs=None)), (1, dict(pt=None)), (1, dict(nkl=None)), (1, dict(npt=None)),
                     (1, dict(pt=(1 << 20) + 2)), (1, dict(npt=(1 << 20) + 4)), (1, dict(nrefs=(4 << 20) + 8)),
                     (1, dict(npt=2 << 20)), (1, dict(nrefs=3 << 20)), (1, dict(nrefs=5 << 20))]:
        assert _resize(lib, **kw) == want, kw


def test_out_of_pages_has_a_name(lib):
    assert fa.fa512_status_string(7) == "FA512_ERR_OUT_OF_PAGES"


def test_bindings_refuse_before_the_library():
    z = torch.zeros
    q, pages = z((1, 4, 8, 512), dtype=torch.bfloat16), z((2, 64, 4, 512), dtype=torch.bfloat16)
    pt, n = z((1, 2), dtype=torch.int32), z(1, dtype=torch.int32)
    bad = [lambda: fa.fa512_decode_paged_tree(q, pages, pages, pt, n),                    # not on a GPU
           lambda: fa.fa512_decode_paged_tree(q[0], pages, pages, pt, n),
           lambda: fa.fa512_decode_paged_tree(q, pages, pages[:1], pt, n),
           lambda: fa.fa512_decode_paged_tree(q, pages, pages, pt, z(2, dtype=torch.int32)),
           lambda: fa.fa512_decode_paged_tree(q, pages, pages, pt, n, z((1, 4, 2), dtype=torch.int32)),
           lambda: fa.fa512_decode_paged_tree(q, pages, pages, pt, n, out=q[:, :2]),
           lambda: fa.fa512_decode_paged_tree_fp8(q, pages, pages, pt, n),
           lambda: fa.fa512_cache_append(q, q, pages, pages, pt, n),                       # 8 heads, 4 in the pages
           lambda: fa.fa512_cache_append(q[:, :, :4], q[:, :, 4:], pages, pages, pt, n),
           lambda: fa.fa512_cache_compact(pages, pages[:1], pt, n, pt, n, q_len=4),
           lambda: fa.fa512_cache_compact(pages.float(), pages.float(), pt, n, pt, n, q_len=4),
           lambda: fa.fa512_cache_fork(pages, pages, pt, n, n, z(3, dtype=torch.int32)),   # pool of 2 pages
           lambda: fa.fa512_cache_resize(pt, n, z(2, dtype=torch.int32), n, page_size=64)]
    for i, f in enumerate(bad):
        with pytest.raises(fa.Fa512Error):
            f()
            pytest.fail("call %d was not refused" % i)


def test_fork_refuses_outputs_that_overlap(lib):
    for kw in (dict(nkl=(5 << 20) + 44), dict(npt=(7 << 20) + 36), dict(nrefs=(6 << 20) + 8)):
        assert _fork(lib, **kw) == 1, kw
