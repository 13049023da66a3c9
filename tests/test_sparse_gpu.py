"""Sparse decode on the GPU: page bounds and the selection exactly, attention over
selected pages within the tolerance below, and the calls of one decode step
together, on a side stream and in a captured graph.

Tolerance of an output element, A = sum p |v| / sum p (fp64): 2^-8 |O| (bf16), the
weights' rounding 2^-8 A (bf16 cache) or 2^-10 A (coded caches, f16) with 2^-24 n
vmax for f16 weights below its normal range, 1e-3 A for the fp32 scores, plus 1e-6.
"""
import numpy as np
import pytest
import torch

from head_dim_flashattention_gb300 import workloads
from oracle import paged

pytestmark = pytest.mark.gpu
D, ROW = 512, 288
KINDS = pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
SCALES = {"bf16": {}, "e4m3": {"k_scale": 0.0371, "v_scale": 0.0517}, "e2m1": {"k_scale": 0.37, "v_scale": 1.3}}


@pytest.fixture(scope="module")
def fa(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    import head_dim_flashattention_gb300 as fa
    fa.load_library()
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def random_cache(shape, kind, seed):
    rng = np.random.RandomState(seed)
    if kind == "bf16":
        return torch.tensor(rng.randn(*shape, D), dtype=torch.float32).to(torch.bfloat16)
    if kind == "e4m3":
        return (torch.tensor(rng.randn(*shape, D), dtype=torch.float32) / 0.04).to(torch.float8_e4m3fn).view(torch.uint8)
    r = rng.randint(0, 256, (*shape, ROW)).astype(np.uint8)
    r[..., 256:] = rng.randint(0x28, 0x32, (*shape, 32))
    return torch.from_numpy(r)


def poison(x, kind, where):
    if kind == "bf16":
        x[where] = float("nan")
    elif kind == "e4m3":
        x[where] = 0x7F
    else:
        x[..., 256:][where] = 0x7F


class Case:
    def __init__(self, lens, q_len, hq, hk, psz, pick, kind, seed):
        rng = np.random.RandomState(seed)
        need = [paged.pages_of(n, psz) for n in lens]
        pool, width = sum(need) + 2, max(1, max(need)) + 1
        perm, at = rng.permutation(pool), 0
        table = np.full((len(lens), width), 1 << 30, dtype=np.int32)
        self.sel = np.full((len(lens), hk, pick), -1, dtype=np.int32)
        for b, k in enumerate(need):
            table[b, :k] = perm[at:at + k]
            at += k
            for h in range(hk):
                some = np.sort(rng.permutation(k)[:min(k, pick)])
                self.sel[b, h, :len(some)] = some
        self.table, self.lens, self.sel = torch.from_numpy(table), i32(lens), torch.from_numpy(self.sel)
        self.k, self.v = random_cache((pool, psz, hk), kind, seed), random_cache((pool, psz, hk), kind, seed + 1)
        self.q = workloads.draft_queries(len(lens), q_len, hq, seed=seed)
        self.kind, self.max_len, self.psz, self.rows = kind, max(lens), psz, q_len * hq // hk

    def poisoned(self):
        """NaN in all that no row sees."""
        seen = torch.zeros(self.k.shape[:3], dtype=torch.bool)
        for b, n in enumerate(self.lens.tolist()):
            for h in range(self.sel.shape[1]):
                for p in self.sel[b, h].tolist():
                    if p >= 0:
                        seen[int(self.table[b, p]), :max(0, min(self.psz, n - p * self.psz)), h] = True
        for x in (self.k, self.v):
            poison(x, self.kind, ~seen)
        return self

    def run(self, fa, dev="cuda", **kw):
        f = {"bf16": fa.fa512_decode_paged_sparse, "e4m3": fa.fa512_decode_paged_sparse_fp8,
             "e2m1": fa.fa512_decode_paged_sparse_fp4}[self.kind]
        c = [x.to(dev) for x in (self.q, self.k, self.v, self.table, self.lens, self.sel)]
        out, lse = f(*c, **{"max_kv_len": self.max_len, **SCALES[self.kind], **kw})
        torch.cuda.synchronize()
        return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)

    def check(self, fa, **kw):
        o, l = self.run(fa, **kw)
        assert fa.fa512_device_status() == 0
        ro, rl, weight = paged.decode_paged_any(self.q, self.k, self.v, self.table, self.lens, self.sel,
                                                **SCALES[self.kind])
        f16 = self.kind != "bf16"
        tol = 2.0 ** -8 * np.abs(ro) + ((2.0 ** -10 if f16 else 2.0 ** -8) + 1e-3) * weight + 1e-6
        if f16:
            tol += 2.0 ** -24 * self.sel.shape[2] * self.psz * 6
        assert np.all(np.isfinite(o))
        worst = np.max(np.abs(o - ro) - tol) if o.size else 0.0
        assert worst <= 0, (worst, np.unravel_index(np.argmax(np.abs(o - ro) - tol), o.shape))
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(l), none) and np.all(o[none] == 0)
        assert np.max(np.abs(l[~none] - rl[~none]), initial=0.0) <= 1e-3
        return o, l


# --------------------------------------------------------------------- bounds

@KINDS
@pytest.mark.parametrize("psz", [16, 64, 256])
@pytest.mark.parametrize("q_len", [1, 5, 130])
def test_bounds(fa, kind, psz, q_len):
    lens, cnts = [q_len, q_len + 60, q_len + 300, 700], [q_len, max(0, q_len - 1), 1, q_len]
    c = Case(lens, 1, 4, 2, psz, 1, kind, 41)
    # what lies behind the sequences' ends is not looked at
    for b, n in enumerate(lens):
        p = (n - 1) // psz
        where = torch.zeros(c.k.shape[:3], dtype=torch.bool)
        where[int(c.table[b, p]), n - p * psz:] = True
        poison(c.k, kind, where)
    before = torch.randn(c.k.shape[0], 2, 2, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    got = fa.fa512_cache_page_bounds(c.k.cuda(), c.table.cuda(), c.lens.cuda(), before.cuda(), q_len=q_len,
                                     q_lens=i32(cnts).cuda())
    want = paged.page_bounds(c.k, c.table, c.lens, before, q_len, i32(cnts))
    assert np.array_equal(paged.widen_bf16(got.cpu()), want)
    assert fa.fa512_device_status() == 0


@KINDS
def test_bounds_of_nan(fa, kind):
    c = Case([40], 1, 4, 2, 64, 1, kind, 42)
    where = torch.zeros(c.k.shape[:3], dtype=torch.bool)
    where[int(c.table[0, 0]), 9, 1] = True
    poison(c.k, kind, where)
    z = torch.zeros(c.k.shape[0], 2, 2, D, dtype=torch.bfloat16).cuda()
    got = fa.fa512_cache_page_bounds(c.k.cuda(), c.table.cuda(), c.lens.cuda(), z, q_len=1).cpu()[int(c.table[0, 0])]
    nan = got[1].isnan()
    assert nan.all() if kind != "e2m1" else nan.any(), "codes of 0 under a NaN scale are NaN too"
    assert not got[0].isnan().any()


def test_bounds_skip_what_lies_outside(fa):
    c = Case([40, 40], 1, 4, 2, 16, 1, "bf16", 43)
    z = torch.zeros(c.k.shape[0], 2, 2, D, dtype=torch.bfloat16)
    for lens, cnts, spoil in (([40, 200], [1, 1], 0), ([40, 1], [1, 2], 0), ([40, 40], [1, 9], 0), ([40, 40], [1, 1], 1)):
        t = c.table.clone()
        if spoil:
            t[1, 2] = -3
        got = fa.fa512_cache_page_bounds(c.k.cuda(), t.cuda(), i32(lens).cuda(), z.cuda(), q_len=4, q_lens=i32(cnts).cuda())
        assert fa.fa512_device_status() == 6
        want = paged.page_bounds(c.k, c.table[:1], i32([40]), z, 1)
        assert np.array_equal(paged.widen_bf16(got.cpu()), want)


# --------------------------------------------------------------------- select

def bounds_of(pool, hk, seed, spread=0.4):
    rng = np.random.RandomState(seed)
    mid = rng.randn(pool, hk, 1, D) * spread
    w = 2.0 + 0.6 * rng.rand(pool, hk, 2, D)
    w[:, :, 0] *= -1
    return torch.tensor(mid + w, dtype=torch.float32).to(torch.bfloat16)


def select_case(lens, q_len, hq, hk, psz, seed):
    need = [paged.pages_of(n, psz) for n in lens]
    pool, width = sum(need) + 2, max(1, max(need)) + 1
    perm, at = np.random.RandomState(seed).permutation(pool), 0
    table = np.full((len(lens), width), -9, dtype=np.int32)
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return workloads.draft_queries(len(lens), q_len, hq, seed=seed), bounds_of(pool, hk, seed), torch.from_numpy(table), i32(lens)


@pytest.mark.parametrize("q_len,hq,hk", [(1, 8, 4), (1, 16, 1), (4, 8, 4), (5, 3, 1), (1, 1, 1), (3, 12, 4)])
@pytest.mark.parametrize("psz,pick,first,last", [(16, 7, 1, 2), (64, 1, 0, 1), (32, 5, 0, 0), (16, 40, 2, 5)])
def test_select(fa, q_len, hq, hk, psz, pick, first, last):
    lens = [1, 16, psz * pick, psz * pick + 1, 1111, 2000, 0]
    q, bounds, table, n = select_case(lens, q_len, hq, hk, psz, 51 + pick)
    got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), n.cuda(), page_size=psz, n_select=pick,
                                max_kv_len=max(lens), n_first=first, n_last=last)
    assert fa.fa512_device_status() == 0
    want = paged.select_pages(q, bounds, table, n, psz, pick, first, last)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("pages", [255, 256, 257, 1025, 5000])
def test_select_among_many(fa, pages):
    q, bounds, table, n = select_case([pages * 16 - 3, 40], 1, 2, 1, 16, 61)
    for pick in (2, 100, pages - 1):
        got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), n.cuda(), page_size=16, n_select=pick)
        assert np.array_equal(got.cpu().numpy(), paged.select_pages(q, bounds, table, n, 16, pick, 1, 1))
    assert fa.fa512_device_status() == 0


def test_equal_scores_go_to_the_lowest_pages(fa):
    q, bounds, table, n = select_case([100 * 16], 1, 2, 1, 16, 62)
    bounds[:] = bounds[0].clone()
    got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), n.cuda(), page_size=16, n_select=9, n_first=0, n_last=1)
    assert got.cpu()[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 99]
    # zeros of either sign are equal
    bounds[:] = 0
    bounds[3:40:2] = -0.0
    got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), n.cuda(), page_size=16, n_select=9, n_first=0, n_last=0)
    assert got.cpu()[0, 0].tolist() == list(range(9))


def test_bounds_that_are_not_finite_come_first(fa):
    q, bounds, table, n = select_case([60 * 16], 1, 2, 1, 16, 63)
    big = int(table[0, 20])
    bounds[big] = 100.0                                  # large
    for i, (p, x) in enumerate([(11, float("nan")), (33, float("inf")), (44, float("-inf"))]):
        bounds[int(table[0, p]), 0, i % 2, 7 + i] = x
    got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), n.cuda(), page_size=16, n_select=4, n_first=0, n_last=1)
    assert got.cpu()[0, 0].tolist() == [11, 33, 44, 59]


@pytest.mark.parametrize("pages", [7, 300, 4500])
def test_scores_that_differ_in_any_bit(fa, pages):
    """Scores that are equal but for one of 32 bits or their sign, and only those always chosen."""
    q, bounds, table, n = select_case([pages * 16], 1, 2, 1, 16, 66)
    q[:] = 0
    q[0, 0, :, 0] = 1.0
    rng = np.random.RandomState(pages)
    value = torch.tensor(np.exp2(rng.randint(-120, 120, pages)) * rng.choice([-1.0, 1.0, 1.0078125], pages),
                         dtype=torch.float32).to(torch.bfloat16)
    bounds[:] = 0
    bounds[table[0, :pages].long(), 0, :, 0] = value[:, None]
    for pick, first, last in ((1, 0, 0), (3, 1, 2), (5, 2, 1), (6, 0, 1), (pages - 1, 1, 1)):
        got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), n.cuda(), page_size=16, n_select=pick,
                                    n_first=first, n_last=last).cpu().numpy()
        assert np.array_equal(got, paged.select_pages(q, bounds, table, n, 16, pick, first, last))
    assert fa.fa512_device_status() == 0


def test_first_and_last_pages_come_before_those_that_are_not_finite(fa):
    q, bounds, table, n = select_case([60 * 16], 1, 4, 2, 16, 65)
    for i, p in enumerate((4, 9, 30, 31, 32, 50)):
        bounds[int(table[0, p]), 1, i % 2, 3 * i] = float("nan") if i % 3 else float("-inf")
    for pick in (3, 5, 7, 12):
        got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), n.cuda(), page_size=16, n_select=pick, n_first=1,
                                    n_last=2).cpu().numpy()
        assert np.array_equal(got, paged.select_pages(q, bounds, table, n, 16, pick, 1, 2))
        assert {0, 58, 59} <= set(got[0, 1].tolist())


def test_select_records_what_lies_outside(fa):
    q, bounds, table, n = select_case([60 * 16, 30 * 16], 1, 2, 1, 16, 64)
    table[0, 5] = 1 << 25
    table[1, 6] = -1
    got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), n.cuda(), page_size=16, n_select=29).cpu()
    assert fa.fa512_device_status() == 6
    assert 5 not in got[0, 0].tolist() and got[1, 0].tolist() == [p for p in range(30) if p != 6]
    got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), i32([60 * 16, -4]).cuda(), page_size=16, n_select=3,
                                max_kv_len=30 * 16).cpu()
    assert fa.fa512_device_status() == 6
    assert got.max() == 29 and got[1, 0].tolist() == [-1, -1, -1]


# --------------------------------------------------------------------- sparse

@KINDS
@pytest.mark.parametrize("psz", [16, 32, 64, 128, 256])
def test_sparse_page_sizes(fa, kind, psz):
    Case([1, 15, 17, 64, 700, 1500], 1, 8, 4, psz, 5, kind, 71).poisoned().check(fa)


@KINDS
@pytest.mark.parametrize("q_len,hq,hk", [(1, 4, 4), (1, 32, 4), (1, 16, 1), (3, 8, 4), (5, 12, 4), (16, 2, 2), (2, 8, 1)])
def test_sparse_rows(fa, kind, q_len, hq, hk):
    Case([900, 33, q_len, 2], q_len, hq, hk, 32, 9, kind, 72).check(fa)


@KINDS
@pytest.mark.parametrize("splits", [1, 2, 5, 200, 1024])
@pytest.mark.parametrize("rows", [2, 12])
def test_sparse_split_counts(fa, kind, splits, rows):
    Case([3000, 65, 0], 1, rows, 1, 16, 70, kind, 73).check(fa, num_splits=splits)


@KINDS
@pytest.mark.parametrize("splits", [0, 1, 6])
@pytest.mark.parametrize("batch,hk", [(33, 3), (150, 2)])
def test_many_ragged_lists(fa, kind, batch, hk, splits):
    rng = np.random.RandomState(batch)
    lens = np.where(rng.rand(batch) < 0.2, 0, rng.randint(1, 500, batch))
    lens[-1] = 900
    Case(lens.tolist(), 2, 4 * hk, hk, 16, 12, kind, 90).poisoned().check(fa, num_splits=splits)


@KINDS
@pytest.mark.parametrize("batch,pick", [(2, 16), (3, 16), (16, 20), (5, 30)])
def test_full_lists_of_equal_length(fa, kind, batch, pick):
    """Ranges that a number of groups for each sequence cuts evenly, and not."""
    Case([600] * batch, 1, 8, 4, 16, pick, kind, 91).poisoned().check(fa)


@KINDS
def test_all_pages_selected_is_the_dense_call(fa, kind):
    c = Case([1000, 130, 64], 1, 8, 4, 64, 16, kind, 74)
    o, l = c.check(fa)
    dense = {"bf16": fa.fa512_decode_paged, "e4m3": fa.fa512_decode_paged_fp8, "e2m1": fa.fa512_decode_paged_fp4}[kind]
    q = c.q[:, 0] if kind == "bf16" else c.q
    do, dl = dense(q.contiguous().cuda(), c.k.cuda(), c.v.cuda(), c.table.cuda(), c.lens.cuda(), max_kv_len=1000, **SCALES[kind])
    tol = 2.0 ** -7 * np.abs(o) + 2e-2
    assert np.all(np.abs(do.float().cpu().numpy().reshape(o.shape) - o) <= tol)
    assert np.allclose(dl.cpu().numpy().reshape(l.shape), l, rtol=0, atol=1e-4)


@KINDS
@pytest.mark.parametrize("rows", [2, 12])
def test_empty_lists_and_lists_of_other_lengths(fa, kind, rows):
    c = Case([1000, 500, 300], 1, rows, 1, 16, 40, kind, 75)
    c.sel[0, 0] = -1
    c.sel[1, 0, 3:] = -1
    c.sel[2, 0] = torch.cat([i32([18]), torch.full((39,), -1, dtype=torch.int32)])   # the page that is filling alone
    o, l = c.poisoned().check(fa)
    assert np.isneginf(l[0]).all() and np.isfinite(l[1:]).all()


@KINDS
@pytest.mark.parametrize("rows", [2, 12])
def test_bad_lists_are_recorded(fa, kind, rows):
    for bad in ([3, 3], [5, 2], [0, 1 << 20], [0, 63], [-1, 4], [2, -1, 2]):
        c = Case([1000], 1, rows, 1, 16, 40, kind, 76)
        c.sel[0, 0] = -1
        c.sel[0, 0, :len(bad)] = i32(bad)
        c.run(fa)
        assert fa.fa512_device_status() == 6, bad
    c = Case([1000], 1, rows, 1, 16, 40, kind, 76)
    c.table[0, int(c.sel[0, 0, 2])] = 1 << 20
    o, _ = c.run(fa)
    assert fa.fa512_device_status() == 6 and np.isfinite(o).all()


@KINDS
@pytest.mark.parametrize("rows", [2, 12])
def test_sparse_nan_scores(fa, kind, rows):
    c = Case([200, 130], 1, rows, 1, 64, 4, kind, 77)
    where = torch.zeros(c.k.shape[:3], dtype=torch.bool)
    where[int(c.table[0, 1]), 7, 0] = True
    poison(c.k, kind, where)
    o, l = c.run(fa)
    assert np.isnan(o[0]).all() and np.isnan(l[0]).all() and np.isfinite(o[1]).all()


@KINDS
@pytest.mark.parametrize("rows", [2, 8, 12])
@pytest.mark.parametrize("shape", ["rising", "falling", "one above many", "one below many", "steps", "far below", "late"])
def test_scores_that_rise_and_fall(fa, kind, rows, shape):
    """The softmax's references rise with the scores, and only now and then: scores set by one channel."""
    n, hk, psz = 3000, 2, 64
    j, rng = np.arange(n), np.random.RandomState(7)
    score = {"rising": 0.02 * j, "falling": 60 - 0.02 * j, "one above many": np.where(j == 5, 0.0, -10.5),
             "one below many": np.where(j == 5, -30.0, 1.0), "steps": rng.randint(-4, 5, n) * 2.0 + 6.0 * (j // 500),
             "far below": -300.0 + 0.01 * j, "late": np.where(j < 2900, -20.0, 0.0)}[shape]
    c = Case([n, 700], rows // 2, 2 * hk, hk, psz, 47, kind, 95)
    c.q[:] = 0
    c.q[..., 0] = 1.0
    x = torch.zeros(*c.k.shape[:3], D)
    for b, m in enumerate((n, 700)):
        x[c.table[b].long()[j[:m] // psz], j[:m] % psz, :, 0] = torch.tensor(score[:m], dtype=torch.float32)[:, None]
    x = x.to(torch.bfloat16)
    c.k = x if kind == "bf16" else torch.from_numpy(paged.fp4_rows(x, 0.37)) if kind == "e2m1" else (
        (x.float() / 0.0371 / 32).to(torch.float8_e4m3fn).view(torch.uint8))
    scale = 1.0 if kind != "e4m3" else 32.0
    o, l = c.run(fa, scale=scale)
    assert fa.fa512_device_status() == 0
    ro, rl, weight = paged.decode_paged_any(c.q, c.k, c.v, c.table, c.lens, c.sel, scale=scale, **SCALES[kind])
    # as in Case.check; f16 weights below its normal range are off by 2^-25 where the largest is above 1
    tol = 2.0 ** -8 * np.abs(ro) + ((2.0 ** -8 if kind == "bf16" else 2.0 ** -10) + 1e-3) * weight + 1e-6
    if kind != "bf16":
        tol += 2.0 ** -24 * n * 6
    assert np.all(np.isfinite(o)) and np.max(np.abs(o - ro) - tol) <= 0
    assert np.max(np.abs(l - rl)) <= 1e-3


@KINDS
def test_sparse_repeats_bitwise(fa, kind):
    c = Case([3000, 700, 64], 1, 8, 4, 64, 9, kind, 78)
    a = c.run(fa)
    for _ in range(3):
        b = c.run(fa)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


# ------------------------------------------------------------- a step together

def step(fa, s, kind, stream=None):
    """One decode step: the new token's rows, the bounds of its page, the pages, the attention."""
    kw = {"stream": stream} if stream is not None else {}
    append = {"bf16": fa.fa512_cache_append, "e4m3": fa.fa512_cache_append_fp8, "e2m1": fa.fa512_cache_append_fp4}[kind]
    attend = {"bf16": fa.fa512_decode_paged_sparse, "e4m3": fa.fa512_decode_paged_sparse_fp8,
              "e2m1": fa.fa512_decode_paged_sparse_fp4}[kind]
    append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], **SCALES[kind], **kw)
    fa.fa512_cache_page_bounds(s["k"], s["table"], s["lens"], s["bounds"], q_len=1, **kw)
    sel = fa.fa512_select_pages(s["q"], s["bounds"], s["table"], s["lens"], page_size=16, n_select=9, max_kv_len=600,
                                n_last=2, **kw)
    return (sel,) + attend(s["q"], s["k"], s["v"], s["table"], s["lens"], sel, max_kv_len=600, **SCALES[kind], **kw)


def state(kind):
    c = Case([600, 333, 20], 1, 8, 4, 16, 9, kind, 81)
    s = {"k": c.k, "v": c.v, "table": c.table, "lens": c.lens, "q": c.q,
         "k_new": workloads.randn_bf16((3, 1, 4, D), 5), "v_new": workloads.randn_bf16((3, 1, 4, D), 6)}
    z = torch.zeros(c.k.shape[0], 4, 2, D, dtype=torch.bfloat16)
    s["bounds"] = torch.tensor(paged.page_bounds(c.k, c.table, c.lens, z, 600, c.lens), dtype=torch.float32).to(torch.bfloat16)
    return s


@KINDS
def test_a_step_eager_on_a_side_stream_and_captured(fa, kind):
    s = state(kind)
    up = lambda: {k: v.cuda() for k, v in s.items()}  # noqa: E731
    d = up()
    sel, out, lse = step(fa, d, kind)
    torch.cuda.synchronize()
    assert fa.fa512_device_status() == 0
    # the step by the references, from the cache it wrote
    k, v = d["k"].cpu(), d["v"].cpu()
    bounds = paged.page_bounds(k, s["table"], s["lens"], s["bounds"], 1)
    assert np.array_equal(paged.widen_bf16(d["bounds"].cpu()), bounds)
    assert np.array_equal(sel.cpu().numpy(), paged.select_pages(s["q"], d["bounds"].cpu(), s["table"], s["lens"], 16, 9, 1, 2))
    ro, rl, weight = paged.decode_paged_any(s["q"], k, v, s["table"], s["lens"], sel.cpu(), **SCALES[kind])
    assert np.all(np.abs(out.float().cpu().numpy() - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 1e-3) * weight + 1e-6)
    assert np.all(np.abs(lse.cpu().numpy() - rl) <= 1e-3)

    side, e = torch.cuda.Stream(), up()
    torch.cuda.synchronize()
    got = step(fa, e, kind, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (sel, out, lse)))

    g, f = torch.cuda.CUDAGraph(), up()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cap = step(fa, f, kind)
    for _ in range(2):
        f["k"].copy_(s["k"].cuda())
        f["bounds"].zero_()
        f["bounds"].copy_(s["bounds"].cuda())
        for x in cap:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cap, (sel, out, lse)))
    # a longer sequence in the same graph
    f["lens"].copy_(i32([599, 340, 33]).cuda())
    f["table"][2, 2] = int(f["table"][0, 37])            # its third page, of another sequence's last
    g.replay()
    torch.cuda.synchronize()
    want = step(fa, {**f, "k": f["k"].clone(), "v": f["v"].clone(), "bounds": f["bounds"].clone()}, kind)
    assert all(torch.equal(a, b) for a, b in zip(cap, want))
    fa.fa512_device_status()


def test_two_captured_steps_with_workspaces_of_their_own(fa):
    """Two graphs that run at once on two streams, each with its own workspace."""
    c = [Case([3000, 2000], 1, 8, 4, 64, 12, "e2m1", 91 + i) for i in range(2)]
    want = [x.run(fa) for x in c]
    graphs = []
    for x in c:
        d = [t.cuda() for t in (x.q, x.k, x.v, x.table, x.lens, x.sel)]
        n = fa.fa512_decode_workspace_bytes_sparse(2, 1, 8, 4, 4, 64, 12, 3000)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = fa.fa512_decode_paged_sparse_fp4(*d, max_kv_len=3000, workspace=ws, **SCALES["e2m1"])
        graphs.append((g, out, d, ws))
    streams = [torch.cuda.Stream() for _ in c]
    for _ in range(5):
        for (g, out, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, out, _, _), w in zip(graphs, want):
            assert np.array_equal(out[0].float().cpu().numpy().astype(np.float64), w[0])
