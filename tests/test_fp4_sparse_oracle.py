"""The references of the 4-bit cache and of selected pages against closed forms,
and the calls' refusals before anything is launched (no GPU)."""
import numpy as np
import pytest
import torch

import __graft_entry__
import head_dim_flashattention_gb300 as fa
from oracle import paged


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return fa.load_library()


def bf16(x):
    return torch.tensor(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def row(values):
    x = np.zeros(512, dtype=np.float32)
    x[:len(values)] = values
    return bf16(x)


# ----------------------------------------------------------------- references

def test_every_pair_of_codes_and_scales_widens():
    rows = np.zeros((256, 288), dtype=np.uint8)
    rows[:, :256] = np.arange(256)                     # every byte of codes
    rows[:, 256:] = np.arange(256)[:, None]            # under every scale
    x = paged.widen_fp4(rows).reshape(256, 256, 2)
    codes = np.concatenate([paged.E2M1, -paged.E2M1])
    from oracle import e4m3_table
    for s in (0, 1, 8, 0x38, 0x7E, 0xB8):
        assert np.array_equal(x[s, :, 0], codes[np.arange(256) % 16] * e4m3_table()[s])
        assert np.array_equal(x[s, :, 1], codes[np.arange(256) // 16] * e4m3_table()[s])
    assert np.isnan(x[0x7F]).all()


def test_values_of_the_format_are_kept():
    """Rows whose groups hold code times scale, with the largest code among them, come back as they were."""
    rng = np.random.RandomState(0)
    from oracle import e4m3_table
    s = e4m3_table()[rng.randint(9, 0x7F, 32)]
    x = np.concatenate([paged.E2M1, -paged.E2M1])[rng.randint(0, 16, (32, 16))] * s[:, None]
    x[:, 3] = 6 * s
    r = paged.fp4_rows(bf16(x.reshape(512)), 1.0)
    assert np.array_equal(paged.widen_fp4(r), x.reshape(512))
    r2 = paged.fp4_rows(bf16(x.reshape(512) / 8), 0.125)
    assert np.array_equal(r, r2)


def test_rounding_of_codes_and_scales():
    # scale 1: the largest is 6; ties go to the even code
    r = paged.fp4_rows(row([6, 0.25, 0.26, 0.75, 0.74, 1.25, 1.75, 2.5, 3.5, 5, 5.1, -0.25, -5.5]), 1.0)
    got = paged.widen_fp4(r)[:13]
    assert got.tolist() == [6, 0, 0.5, 1, 0.5, 1, 2, 2, 4, 4, 6, 0, -6]
    assert r[256] == 0x38 and r[257:].max() == 0
    # beyond the largest scale, infinities, NaN, what is too small
    assert paged.widen_fp4(paged.fp4_rows(row([1e6, 3.0]), 1.0))[:2].tolist() == [2688, 0]
    assert paged.widen_fp4(paged.fp4_rows(row([-np.inf, 448.0]), 1.0))[:2].tolist() == [-2688, 448]
    assert np.isnan(paged.widen_fp4(paged.fp4_rows(row([np.nan, 1.0]), 1.0))[:16]).all()
    assert not paged.fp4_rows(row([6 * 2.0 ** -10, 1e-9]), 1.0).any()      # a tie, to the even scale 0
    assert paged.fp4_rows(row([7 * 2.0 ** -10]), 1.0)[256] == 1


def test_attention_over_one_format_or_another():
    """Values that all formats hold: the same attention; selecting all pages: the dense one."""
    rng = np.random.RandomState(1)
    psz, hk = 16, 2
    x = np.concatenate([paged.E2M1, -paged.E2M1])[rng.randint(0, 16, (2, 5, psz, hk, 512))]
    x[..., ::16] = 6
    k16, v16 = bf16(x[0]), bf16(x[1])
    k4, v4 = (torch.from_numpy(paged.fp4_rows(t, 1.0)) for t in (k16, v16))
    k8, v8 = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (k16, v16))
    q = bf16(rng.randn(2, 3, 4, 512))
    pt, kl = np.array([[3, 1, 0], [2, 4, -7]], dtype=np.int32), np.array([40, 17], dtype=np.int32)
    want = paged.decode_paged_tree(q, k16, v16, pt, kl)
    for k, v in ((k16, v16), (k8, v8), (k4, v4)):
        for sel in (None, np.tile(np.array([0, 1, 2, -1]), (2, 2, 1))):
            if sel is not None:
                sel = np.where(sel < np.array([3, 2])[:, None, None], sel, -1)
            got = paged.decode_paged_any(q, k, v, pt, kl, sel)
            assert all(np.allclose(a, b, rtol=1e-12, atol=1e-12) for a, b in zip(got, want))
    one = paged.decode_paged_any(q[:, :1], k4, v4, pt, np.array([1, 1], dtype=np.int32))
    assert np.array_equal(one[0][:, 0, 0], x[1][[3, 2], 0, 0])             # one key: its value


def test_bounds_hold_and_the_largest_are_chosen():
    rng = np.random.RandomState(2)
    psz, hk, pool = 16, 2, 12
    k = bf16(rng.randn(pool, psz, hk, 512) * np.exp(rng.randn(pool, 1, 1, 1)))
    pt, kl = np.arange(10, dtype=np.int32)[None], np.array([150], dtype=np.int32)
    bounds = bf16(paged.page_bounds(k, pt, kl, torch.zeros(pool, hk, 2, 512, dtype=torch.bfloat16), 150))
    q = bf16(rng.randn(1, 1, 4, 512))
    score = paged.page_scores(q, bounds, pt, kl, 0, psz)
    kf, qf = paged.widen_bf16(k), paged.widen_bf16(q)
    for h in range(hk):
        for p in range(10):
            n = min(psz, 150 - p * psz)
            assert (qf[0, 0, 2 * h:2 * h + 2] @ kf[p, :n, h].T).max() <= score[h, p] * (1 + 1e-12)
    got = paged.select_pages(q, bounds, pt, kl, psz, 5, 1, 2)
    for h in range(hk):
        assert {0, 8, 9} <= set(got[0, h])
        mid = score[h, 1:8]
        assert set(got[0, h]) - {0, 8, 9} == set(1 + np.argsort(-mid)[:2])
    assert paged.select_pages(q, bounds, pt, kl, psz, 12, 1, 2)[0, 0].tolist() == list(range(10)) + [-1, -1]
    bounds[2:8, 1, 0, 5] = float("inf")                  # before the others, but for the first and the last
    assert paged.select_pages(q, bounds, pt, kl, psz, 5, 1, 2)[0, 1].tolist() == [0, 2, 3, 8, 9]


# ------------------------------------------------------- refusals before a launch

INF, NAN = float("inf"), float("nan")


def _fp4(lib, **kw):
    a = dict(q=16, kp=16, vp=16, pt=16, kl=16, out=16, lse=None, b=2, qlen=1, hq=8, hk=4, ps=64, npages=10, mpps=4,
             maxlen=200, scale=0.05, ks=0.1, vs=0.1, window=0, splits=2, ws=256, wsb=1 << 30)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.fa512_decode_paged_fp4(*a.values(), None)


def _sparse(lib, bits=16, **kw):
    a = dict(q=16, kp=16, vp=16, pt=16, kl=16, sel=16, out=16, lse=None, b=2, qlen=1, hq=8, hk=4, ps=64, npages=10,
             mpps=4, nsel=3, maxlen=200, scale=0.05, ks=0.1, vs=0.1, splits=2, ws=256, wsb=1 << 30)
    assert set(kw) <= set(a)
    a.update(kw)
    if bits == 16:
        del a["ks"], a["vs"]
    name = {16: "fa512_decode_paged_sparse", 8: "fa512_decode_paged_sparse_fp8", 4: "fa512_decode_paged_sparse_fp4"}
    return getattr(lib, name[bits])(*a.values(), None)


DECODE = [(1, dict(b=-1)), (1, dict(qlen=0)), (1, dict(hq=6)), (1, dict(hk=0)), (1, dict(npages=0)), (1, dict(mpps=0)),
          (1, dict(maxlen=300)), (1, dict(maxlen=-1)), (1, dict(splits=-1)), (1, dict(splits=2000)),
          (1, dict(scale=NAN)), (1, dict(scale=INF)), (1, dict(q=None)), (1, dict(pt=None)), (1, dict(kl=None)),
          (1, dict(out=None)), (1, dict(kp=None)), (1, dict(q=8)), (1, dict(kp=24)), (1, dict(vp=20)), (1, dict(out=40)),
          (1, dict(lse=2)), (1, dict(pt=18)), (2, dict(hq=68)), (2, dict(qlen=9)), (2, dict(qlen=1 << 30)), (2, dict(ps=48)),
          (2, dict(npages=1 << 24, ps=256)), (2, dict(b=65536)), (2, dict(b=65535, qlen=2)), (5, dict(ws=None)),
          (5, dict(wsb=1000)), (5, dict(ws=272)), (0, dict(b=0, q=None))]


def test_fp4_decode_refusals(lib):
    for want, kw in DECODE + [(1, dict(ks=INF)), (1, dict(vs=NAN)), (2, dict(mpps=1 << 25, ps=64)),
                              (2, dict(b=30000, mpps=1 << 20, ps=256, maxlen=1 << 28, splits=1))]:
        assert _fp4(lib, **kw) == want, kw


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_sparse_refusals(lib, bits):
    more = [(1, dict(nsel=0)), (1, dict(nsel=-3)), (1, dict(sel=None)), (1, dict(sel=18)), (2, dict(nsel=1 << 26)),
            (2, dict(mpps=1 << 25, ps=64)),
            (2, dict(b=30000, mpps=1 << 20, ps=256, maxlen=1 << 28, nsel=1 << 20, splits=1))]
    for want, kw in DECODE + more + ([(1, dict(ks=INF)), (1, dict(vs=NAN))] if bits != 16 else []):
        assert _sparse(lib, bits, **kw) == want, kw


def test_fp4_append_refusals(lib):
    def call(**kw):
        a = dict(kn=16, vn=16, kb=2048, kt=2048, vb=2048, vt=2048, kp=16, vp=16, pt=16, kl=16, ql=None, ks=0.1, vs=0.1,
                 b=2, qlen=4, hk=4, ps=64, npages=10, mpps=4)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.fa512_cache_append_fp4(*a.values(), None)
    for want, kw in [(1, dict(b=-1)), (1, dict(qlen=-1)), (1, dict(hk=0)), (1, dict(npages=0)), (1, dict(mpps=0)),
                     (1, dict(kb=12)), (1, dict(vt=4)), (1, dict(ks=0.0)), (1, dict(vs=-1.0)), (1, dict(ks=INF)),
                     (1, dict(vs=NAN)), (1, dict(kn=None)), (1, dict(vp=None)), (1, dict(kn=8)), (1, dict(vp=24)),
                     (1, dict(ql=2)), (2, dict(ps=48)), (2, dict(b=65536)), (2, dict(mpps=1 << 26)),
                     (2, dict(qlen=1 << 28)), (0, dict(b=0, kn=None)), (0, dict(qlen=0, kn=None))]:
        assert call(**kw) == want, kw


def test_bounds_refusals(lib):
    def call(**kw):
        a = dict(kp=16, pt=16, kl=16, ql=None, bounds=16, b=2, qlen=4, hk=4, bits=16, ps=64, npages=10, mpps=4)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.fa512_cache_page_bounds(*a.values(), None)
    for want, kw in [(1, dict(b=-1)), (1, dict(qlen=-1)), (1, dict(hk=0)), (1, dict(bits=32)), (1, dict(bits=0)),
                     (1, dict(npages=0)), (1, dict(mpps=0)), (1, dict(kp=None)), (1, dict(bounds=None)),
                     (1, dict(kl=None)), (1, dict(kp=8)), (1, dict(bounds=24)), (1, dict(ql=3)), (1, dict(pt=2)),
                     (2, dict(ps=48)), (2, dict(b=65536)), (2, dict(hk=65536)), (2, dict(mpps=1 << 26)),
                     (2, dict(hk=65535, qlen=1 << 30, mpps=1 << 22)), (0, dict(b=0, kp=None)), (0, dict(qlen=0, kp=None))]:
        assert call(**kw) == want, kw


def test_select_refusals(lib):
    def call(**kw):
        a = dict(q=16, bounds=16, pt=16, kl=16, sel=16, b=2, qlen=1, hq=8, hk=4, ps=64, npages=10, mpps=4, maxlen=200,
                 nsel=3, first=1, last=1, ws=256, wsb=1 << 20)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.fa512_select_pages(*a.values(), None)
    for want, kw in [(1, dict(b=-1)), (1, dict(qlen=0)), (1, dict(hq=6)), (1, dict(hk=0)), (1, dict(npages=0)),
                     (1, dict(mpps=0)), (1, dict(maxlen=-1)), (1, dict(maxlen=300)), (1, dict(nsel=0, first=0, last=0)),
                     (1, dict(first=-1)), (1, dict(last=-1)), (1, dict(first=2, last=2)),
                     (1, dict(first=1 << 30, last=1 << 30, nsel=1 << 30)), (1, dict(q=None)), (1, dict(sel=None)),
                     (1, dict(q=8)), (1, dict(bounds=20)), (1, dict(sel=2)), (2, dict(hq=68)), (2, dict(qlen=9)),
                     (2, dict(ps=7)), (2, dict(b=65536)), (2, dict(mpps=1 << 25)), (5, dict(ws=None)), (5, dict(wsb=16)),
                     (5, dict(ws=128)), (0, dict(b=0, q=None))]:
        assert call(**kw) == want, kw


def test_sizes_of_workspaces(lib):
    w, s = fa.fa512_decode_workspace_bytes_fp4, fa.fa512_decode_auto_splits_fp4
    rows = 4 * 2 * 8 * 3
    assert w(4, 2, 8, 4, 64, 4096, 3) == rows * 2048 + (rows * 8 + 255) // 256 * 256
    for b, n in ((1, 4096), (16, 16384), (64, 28672)):
        k = s(b, 1, 8, 4, 64, n)
        assert 1 <= k <= n // 64 and w(b, 1, 8, 4, 64, n) == w(b, 1, 8, 4, 64, n, k)
    assert s(1, 1, 8, 4, 64, 0) == 1 and s(0, 1, 8, 4, 64, 100) == 1
    for bad in ((-1, 1, 8, 4, 64, 100, 0), (1, 0, 8, 4, 64, 100, 0), (1, 1, 6, 4, 64, 100, 0), (1, 9, 8, 4, 64, 100, 0),
                (1, 1, 8, 4, 64, -1, 0), (1, 1, 8, 4, 64, 100, 2000), (65535, 2, 8, 4, 64, 100, 1)):
        assert w(*bad) == 0, bad
    wp = fa.fa512_decode_workspace_bytes_sparse
    for bits in (16, 8, 4):
        k = fa.fa512_decode_auto_splits_sparse(16, 1, 8, 4, bits, 64, 37, 28672)
        assert 1 <= k <= 37 * 2 and wp(16, 1, 8, 4, bits, 64, 37, 28672) == wp(16, 1, 8, 4, bits, 64, 37, 28672, k)
        # a list longer than the sequence asks for no more than the sequence
        assert wp(16, 1, 8, 4, bits, 64, 10 ** 6, 640) == wp(16, 1, 8, 4, bits, 64, 10, 640)
    assert wp(16, 1, 8, 4, 5, 64, 37, 28672) == 0 and wp(16, 1, 8, 4, 16, 48, 37, 28672) == 0
    assert wp(16, 1, 8, 4, 16, 64, 0, 28672) == 0
    ws = fa.fa512_select_workspace_bytes
    assert ws(3, 4, 64, 6401) == (3 * 4 * 101 * 4 + 255) // 256 * 256 and ws(0, 4, 64, 100) == 256
    assert ws(-1, 4, 64, 10) == 0 and ws(1, 0, 64, 10) == 0 and ws(1, 1, 48, 10) == 0 and ws(1, 1, 64, -1) == 0


def test_compact_and_fork_take_4_bit_rows_and_nothing_else_new(lib):
    for eb, want in ((-4, 0), (0, 1), (4, 1), (-1, 1)):
        assert lib.fa512_cache_compact(16, 16, 16, 16, None, 16, 16, 1 << 20, 1, 0, 4, 3, 4, eb, 64, 10, 4, None) == want
        if want:
            assert lib.fa512_cache_fork(16, 16, 16, 16, 16, 16, 16, 16, 16, 1, 2, 2, 4, eb, 64, 10, 4, None) == want


def test_the_binding_refuses_before_it_launches():
    x = torch.zeros(1)
    with pytest.raises(fa.Fa512Error):
        fa.fa512_decode_paged_sparse(x, x, x, x, x, None)
    with pytest.raises(fa.Fa512Error):
        fa.fa512_decode_paged_fp4(x.view(1, 1, 1), x.view(1, 1, 1, 1), x, x.view(1, 1), x)
    with pytest.raises(fa.Fa512Error):
        fa.fa512_select_pages(x.view(1, 1, 1), x, x, x, page_size=64, n_select=3)
    with pytest.raises(fa.Fa512Error):
        fa.fa512_cache_page_bounds(x.view(1, 1, 1, 1), x.view(1, 1), x, x, q_len=1)


def test_caches_without_dimensions_are_refused():
    x, z = torch.zeros(1), torch.zeros(())
    t, n = torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for f in (lambda: fa.fa512_cache_compact(z, z, t, n, t, n, q_len=1),
              lambda: fa.fa512_cache_fork(z, z, t, n, n, x),
              lambda: fa.fa512_cache_page_bounds(z, t, n, x, q_len=1),
              lambda: fa.fa512_cache_append_fp4(z, z, z, z, t, n),
              lambda: fa.fa512_decode_paged_fp4(z, z, z, t, n),
              lambda: fa.fa512_select_pages(z, z, t, n, page_size=64, n_select=1)):
        with pytest.raises(fa.Fa512Error):
            f()


def test_sizes_for_pages_that_no_call_takes(lib):
    for psz in (0, -64, 8, 48, 512):
        assert fa.fa512_decode_workspace_bytes_fp4(1, 1, 8, 4, psz, 4096) == 0
        assert fa.fa512_decode_auto_splits_fp4(1, 1, 8, 4, psz, 4096) == 1
        assert fa.fa512_decode_workspace_bytes_sparse(1, 1, 8, 4, 16, psz, 9, 4096) == 0
        assert fa.fa512_decode_auto_splits_sparse(1, 1, 8, 4, 16, psz, 9, 4096) == 1
