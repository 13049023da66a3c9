"""The 4-bit cache on the GPU: append, decode, compact and fork against the plain
references.  Codes and scales are compared exactly.

Tolerance of an output element, with A = sum p |v| / sum p of its row (fp64):
  2^-8 |O|      the output's rounding to bf16 (half a step),
  2^-10 A       each weight's rounding to f16 and, for up to 2 rows a KV head, its
                product's with a group scale (half a step each),
  2^-24 n vmax  n weights below f16's normal range, off by at most 2^-25 of the
                largest one, which is above 1/2 of its tile's reference,
  1e-3 A        the scores: queries and keys are exact in f16, the 512 products
                of a score are summed in fp32, off by at most 512 * 2^-24 * 2 of
                sum |q k| scale, which is below 16 for values of size 1,
plus 1e-6.  LSE: 1e-3.
"""
import numpy as np
import pytest
import torch

from head_dim_flashattention_gb300 import workloads
from oracle import paged

pytestmark = pytest.mark.gpu
D, ROW = 512, 288


@pytest.fixture(scope="module")
def fa(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    import head_dim_flashattention_gb300 as fa
    fa.load_library()
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def tables(lens, psz, width, pool, seed, spare_entry=1 << 30):
    perm = np.random.RandomState(seed).permutation(pool)
    t = np.full((len(lens), width), spare_entry, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = paged.pages_of(n, psz)
        t[b, :k] = perm[at:at + k]
        at += k
    return torch.from_numpy(t)


def random_rows(shape, seed):
    """4-bit rows of plausible scales and any codes."""
    rng = np.random.RandomState(seed)
    r = rng.randint(0, 256, (*shape, ROW)).astype(np.uint8)
    r[..., 256:] = rng.randint(0x28, 0x32, (*shape, 32))      # 0.25 .. 0.5625: values up to 3.4
    return torch.from_numpy(r)


class Case:
    """A cache in 4 bits whose slots behind the sequences hold NaN scales."""

    def __init__(self, lens, q_len, hq, hk, psz, seed, window=0, poison=True):
        width = max(1, max(paged.pages_of(n, psz) for n in lens)) + 1
        pool = sum(paged.pages_of(n, psz) for n in lens) + 3
        self.k, self.v = random_rows((pool, psz, hk), seed), random_rows((pool, psz, hk), seed + 1)
        self.table, self.lens = tables(lens, psz, width, pool, seed), i32(lens)
        self.q = workloads.draft_queries(len(lens), q_len, hq, seed=seed)
        self.window, self.max_len = window, max(lens)
        if poison:
            seen = torch.zeros(pool, psz, dtype=torch.bool)
            for b, n in enumerate(lens):
                lo = max(0, n - q_len + 1 - window) if window > 0 else 0
                j = torch.arange(lo, n)
                seen[self.table[b].long()[j // psz], j % psz] = True
            for x in (self.k, self.v):
                x[..., 256:][~seen] = 0x7F

    def run(self, fa, **kw):
        c = [x.cuda() for x in (self.q, self.k, self.v, self.table, self.lens)]
        kw = {"k_scale": 0.37, "v_scale": 1.3, "max_kv_len": self.max_len, "window": self.window, **kw}
        out, lse = fa.fa512_decode_paged_fp4(*c, **kw)
        torch.cuda.synchronize()
        assert fa.fa512_device_status() == 0
        return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)

    def want(self, **kw):
        return paged.decode_paged_any(self.q, self.k, self.v, self.table, self.lens, window=self.window,
                                      **{"k_scale": 0.37, "v_scale": 1.3, **kw})

    def check(self, fa, **kw):
        got = self.run(fa, **kw)
        compare(got, self.want(), int(self.lens.max()), 3.4 * 1.3)
        return got


def compare(got, want, n, vmax, p_half=2.0 ** -10):
    (o, l), (ro, rl, weight) = got, want
    assert np.all(np.isfinite(o))
    tol = 2.0 ** -8 * np.abs(ro) + (p_half + 1e-3) * weight + 2.0 ** -24 * n * vmax + 1e-6
    worst = np.max(np.abs(o - ro) - tol) if o.size else 0.0
    assert worst <= 0, (worst, np.unravel_index(np.argmax(np.abs(o - ro) - tol), o.shape))
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(l), none)
    assert np.all(o[none] == 0)
    assert np.max(np.abs(l[~none] - rl[~none]), initial=0.0) <= 1e-3


# --------------------------------------------------------------------- append

@pytest.mark.parametrize("ks,vs", [(1.0, 0.125), (0.0371, 0.0517)])
@pytest.mark.parametrize("q_len,hk,psz", [(1, 4, 64), (3, 1, 16), (70, 3, 32), (300, 2, 256)])
def test_append_writes_the_nearest_values(fa, q_len, hk, psz, ks, vs):
    lens, cnts = [q_len, q_len + 45, q_len + 301], [q_len, max(1, q_len - 1), (q_len + 1) // 2]
    width = max(paged.pages_of(n, psz) for n in lens)
    pool = sum(paged.pages_of(n, psz) for n in lens) + 2
    table = tables(lens, psz, width, pool, 5)
    rng = np.random.RandomState(q_len)
    # a fused projection's output: strided heads; values over many binades, ties among them
    x = rng.randn(3, q_len, 8, D) * np.exp2(rng.randint(-12, 12, (3, q_len, 8, D // 16)).repeat(16, -1))
    x[:, :, :, ::3] = np.round(x[:, :, :, ::3] * 4) / 4
    qkv = torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)
    k_new, v_new = qkv[:, :, :hk], qkv[:, :, hk:2 * hk]
    old = torch.from_numpy(rng.randint(0, 256, (pool, psz, hk, ROW)).astype(np.uint8))
    dev = qkv.cuda()
    k, v = old.cuda(), old.cuda()
    fa.fa512_cache_append_fp4(dev[:, :, :hk], dev[:, :, hk:2 * hk], k, v, table.cuda(), i32(lens).cuda(),
                              q_lens=i32(cnts).cuda(), k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert fa.fa512_device_status() == 0
    for new, got, s in ((k_new, k, ks), (v_new, v, vs)):
        rows, want = paged.fp4_rows(new, s), old.numpy().copy()
        for b, (n, t) in enumerate(zip(lens, cnts)):
            pos = np.arange(n - t, n)
            want[table[b].numpy()[pos // psz], pos % psz] = rows[b, :t]
        assert np.array_equal(got.cpu().numpy(), want)


def test_append_of_values_that_have_no_nearest(fa):
    x = torch.randn(1, 4, 1, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[0, 0, 0, 5], x[0, 1, 0, 40], x[0, 2, 0, 100], x[0, 3] = float("nan"), float("inf"), float("-inf"), 0
    x[0, 3, 0, 17] = -0.0
    k, v = (torch.zeros(1, 16, 1, ROW, dtype=torch.uint8).cuda() for _ in range(2))
    fa.fa512_cache_append_fp4(x.cuda(), x.cuda(), k, v, i32([[0]]).cuda(), i32([4]).cuda())
    got, want = paged.widen_fp4(k.cpu())[0, :4], paged.widen_fp4(paged.fp4_rows(x, 1.0))[0]
    assert np.isnan(got[0, 0, :16]).all() and np.array_equal(got, want, equal_nan=True)
    assert got[1, 0, 40] == 2688 and got[2, 0, 100] == -2688 and not got[3].any()
    assert np.array_equal(k.cpu().numpy(), v.cpu().numpy())
    # the same bytes as the oracle's, also with scales that are no powers of two
    for s in (1.0, 0.7):
        fa.fa512_cache_append_fp4(x.cuda(), x.cuda(), k, v, i32([[0]]).cuda(), i32([4]).cuda(), k_scale=s, v_scale=s)
        want = paged.fp4_rows(x, s)[0]
        nan = (want[..., 256:] & 0x7f) == 0x7f           # their codes mean nothing, and are 0
        want[..., :256] *= ~nan.repeat(8, -1)
        assert np.array_equal(k.cpu().numpy()[0, :4], want)


def test_append_skips_what_lies_outside(fa):
    """Counts, positions and pages outside their ranges are recorded and not written."""
    x = torch.ones(1, 2, 1, D, dtype=torch.bfloat16).cuda()
    for table, n, cnt in (([[5, 0]], 2, 2), ([[-1, 0]], 2, 2), ([[0, 1]], 33, 1), ([[0, 1]], 1, 2), ([[0, 1]], 9, 3)):
        k, v = (torch.zeros(3, 16, 1, ROW, dtype=torch.uint8).cuda() for _ in range(2))
        fa.fa512_cache_append_fp4(x, x, k, v, i32(table).cuda(), i32([n]).cuda(), q_lens=i32([cnt]).cuda())
        assert fa.fa512_device_status() == 6
        rows = int((k != 0).any(-1).sum())
        assert rows == (1 if (n, cnt) == (1, 2) else 0) and torch.equal(k, v)


# --------------------------------------------------------------------- decode

@pytest.mark.parametrize("psz", [16, 32, 64, 128, 256])
def test_page_sizes_and_lengths(fa, psz):
    Case([1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 641, 1500], 1, 8, 4, psz, 11).check(fa)


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (8, 4), (32, 4), (12, 4), (16, 1), (9, 1), (7, 7)])
def test_head_groupings(fa, hq, hk):
    Case([300, 45, 1025], 1, hq, hk, 64, 12).check(fa)


@pytest.mark.parametrize("q_len,hq,hk", [(2, 8, 4), (4, 8, 4), (5, 8, 4), (8, 8, 4), (16, 4, 4), (3, 5, 1), (2, 8, 1)])
def test_several_tokens(fa, q_len, hq, hk):
    c = Case([q_len, q_len + 1, 700, 64, 1], q_len, hq, hk, 32, 13)
    o, l = c.check(fa)
    assert np.isneginf(l[4, :q_len - 1]).all() and np.isfinite(l[4, q_len - 1]).all()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 63, 64, 65, 200, 4000])
@pytest.mark.parametrize("q_len", [1, 3])
def test_windows(fa, window, q_len):
    Case([900, 77, 64, 3], q_len, 8, 4, 64, 14, window).check(fa)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64, 1024])
def test_split_counts(fa, splits):
    Case([2000, 64, 1, 0], 1, 8, 4, 64, 15).check(fa, num_splits=splits)


def test_long_and_empty_sequences(fa):
    c = Case([0, 20011, 0], 1, 8, 4, 64, 16)
    o, l = c.check(fa)
    assert not o[0].any() and np.isneginf(l[0]).all()


@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("batch,hk", [(33, 3), (160, 4), (400, 1)])
def test_many_ragged_sequences(fa, batch, hk, splits):
    rng = np.random.RandomState(batch)
    lens = np.where(rng.rand(batch) < 0.2, 0, rng.randint(1, 400, batch))
    lens[batch // 2:batch // 2 + 35] = 0                 # more than a warp's worth without a tile
    lens[-1] = 1500
    c = Case(lens.tolist(), 1, 2 * hk, hk, 16, 17)
    c.check(fa, num_splits=splits)
    c.check(fa, num_splits=splits, max_kv_len=c.table.shape[1] * 16)     # a loose bound


@pytest.mark.parametrize("splits", [0, 33, 70, 1024])
def test_many_rows_some_of_many_segments(fa, splits):
    Case([8000] + [17] * 70 + [0], 1, 8, 4, 64, 23).check(fa, num_splits=splits)


def test_more_kv_heads_than_ctas(fa):
    Case([70, 5, 0], 1, 310, 310, 32, 18).check(fa)


def test_sequences_that_share_their_pages(fa):
    c = Case([500, 500, 500], 2, 8, 4, 32, 19, poison=False)
    c.table[1] = c.table[0]
    c.table[2, :7] = c.table[0, :7]
    c.check(fa)


def test_two_calls_at_once(fa):
    cases = [Case([3000, 77], 1, 8, 4, 64, 20 + i) for i in range(2)]
    want = [c.run(fa) for c in cases]
    dev = [[x.cuda() for x in (c.q, c.k, c.v, c.table, c.lens)] for c in cases]
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(fa.fa512_decode_paged_fp4(*dev[i], k_scale=0.37, v_scale=1.3, max_kv_len=3000))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o, l in got[i]:
            assert np.array_equal(o.float().cpu().numpy(), want[i][0]) and np.array_equal(l.cpu().numpy(), want[i][1])


def test_the_same_bits_every_time(fa):
    c = Case([1000, 2049, 3], 2, 8, 4, 64, 17)
    a = c.run(fa)
    for _ in range(3):
        b = c.run(fa)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_scales_and_sizes_of_queries(fa):
    """A tensor scale is a factor of scores and outputs; queries of any size (a power of two is exact)."""
    c = Case([500, 65], 1, 8, 4, 64, 18)
    o, l = c.run(fa, k_scale=0.5, v_scale=0.25)
    q = c.q
    for e in (-100, 70):
        c.q = (q.float() * 2.0 ** e).to(torch.bfloat16)
        o2, l2 = c.run(fa, k_scale=0.5, v_scale=0.5, scale=D ** -0.5 * 2.0 ** -e)
        assert np.array_equal(o2, 2 * o) and np.allclose(l2, l, rtol=0, atol=1e-5)


def test_rising_scores_and_one_key_that_dominates(fa):
    """References that grow from tile to tile, and a late key that outweighs all others: O is its value row."""
    c = Case([640], 1, 2, 1, 64, 19, poison=False)
    c.q = torch.full((1, 1, 2, D), 0.5, dtype=torch.bfloat16)
    x = np.zeros((640, D))
    x[:] = np.arange(640)[:, None] / 256
    rows = torch.from_numpy(paged.fp4_rows(torch.tensor(x, dtype=torch.float32).to(torch.bfloat16), 1.0))
    j = torch.arange(640)
    c.k[c.table[0].long()[j // 64], j % 64, 0] = rows
    c.check(fa, num_splits=1)
    late = rows.clone()
    late[555] = torch.from_numpy(paged.fp4_rows(torch.full((D,), 80.0, dtype=torch.bfloat16), 1.0))
    c.k[c.table[0].long()[j // 64], j % 64, 0] = late
    for splits in (1, 4):
        o, _ = c.run(fa, num_splits=splits, k_scale=1.0, v_scale=1.0)
        row = paged.widen_fp4(c.v[c.table[0, 555 // 64].long(), 555 % 64, 0])
        assert np.array_equal(o[0, 0, 0], row) and np.array_equal(o[0, 0, 1], row)   # 6 bits: exact in bf16


def test_visible_nan_and_infinite_scores(fa):
    for where in ("k", "q", "v"):
        c = Case([200, 130], 1, 2, 1, 64, 20)
        if where == "k":
            c.k[c.table[0, 2].long(), 7, 0, 256 + 3] = 0x7F
        elif where == "v":
            c.v[c.table[0, 2].long(), 7, 0, 256 + 3] = 0x7F
        else:
            c.q[0, 0, 0, 9] = float("inf")
        for splits in (1, 3):
            d = [x.cuda() for x in (c.q, c.k, c.v, c.table, c.lens)]
            o, l = fa.fa512_decode_paged_fp4(*d, max_kv_len=200, num_splits=splits)
            o, l = o.float().cpu(), l.cpu()
            if where == "k":
                assert o[0].isnan().all() and l[0].isnan().all()
            elif where == "v":
                assert o[0, ..., 48:64].isnan().all() and not o[0, ..., :48].isnan().any() and not o[0, ..., 64:].isnan().any()
            else:
                assert o[0, 0, 0].isnan().all() and not o[0, 0, 1].isnan().any()
            assert not o[1].isnan().any() and not l[1].isnan().any()


def test_a_sequence_that_sees_nan_only(fa):
    c = Case([1, 5], 1, 2, 1, 64, 21, poison=False)
    c.k[..., 256:] = 0x7F
    d = [x.cuda() for x in (c.q, c.k, c.v, c.table, c.lens)]
    o, l = fa.fa512_decode_paged_fp4(*d, max_kv_len=64)
    assert o.isnan().all() and l.isnan().all()


def test_bad_pages_and_lengths_are_recorded(fa):
    c = Case([300, 300], 1, 8, 4, 64, 22)
    c.table[0, 1], c.table[1, 0] = 1 << 20, -1
    d = [x.cuda() for x in (c.q, c.k, c.v, c.table, c.lens)]
    o, _ = fa.fa512_decode_paged_fp4(*d, max_kv_len=300)
    assert fa.fa512_device_status() == 6 and o.isfinite().all()
    c = Case([300, 64], 1, 8, 4, 64, 22)
    d = [x.cuda() for x in (c.q, c.k, c.v, c.table, c.lens)]
    o, _ = fa.fa512_decode_paged_fp4(*d, max_kv_len=128)       # the first 128 positions are read
    assert fa.fa512_device_status() == 6 and o.isfinite().all()
    d[4] = i32([-5, 64]).cuda()
    o, l = fa.fa512_decode_paged_fp4(*d, max_kv_len=128)
    assert fa.fa512_device_status() == 6 and l[0].isneginf().all() and l[1].isfinite().all()


def test_pages_beyond_32_bits_of_bytes(fa):
    """Rows whose byte offsets pass 2^32."""
    psz, hk, pool = 256, 4, 15000                              # 4.4 GB
    k, v = (torch.zeros(pool, psz, hk, ROW, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = Case([700], 1, 8, hk, psz, 23, poison=False)
    far = torch.tensor([[14999, 14998, 7500]], dtype=torch.int32)
    for small, big in ((c.k, k), (c.v, v)):
        for i in range(3):
            big[int(far[0, i])] = small[int(c.table[0, i])].cuda()
    want = c.run(fa)
    out, lse = fa.fa512_decode_paged_fp4(c.q.cuda(), k, v, far.cuda(), c.lens.cuda(), k_scale=0.37, v_scale=1.3,
                                         max_kv_len=700)
    assert np.array_equal(out.float().cpu().numpy().astype(np.float64), want[0])
    new = torch.randn(1, 1, hk, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    fa.fa512_cache_append_fp4(new.cuda(), new.cuda(), k, v, far.cuda(), i32([2]).cuda())
    assert np.array_equal(k[14999, 1].cpu().numpy(), paged.fp4_rows(new, 1.0)[0, 0])
    assert fa.fa512_device_status() == 0


# -------------------------------------------------------------- compact, fork

def test_compact_moves_4_bit_rows(fa):
    psz, hk, layers = 16, 3, 2
    lens, cnts = [40, 70, 17], [9, 12, 4]
    pool = 12
    table = tables(lens, psz, 5, pool, 31)
    k = torch.from_numpy(np.random.RandomState(4).randint(0, 256, (layers, pool, psz, hk, ROW)).astype(np.uint8))
    acc = i32([[0, 2, 5, 8], [3, 4, 11, -1], [0, 1, 2, 3]])
    n = i32([4, 3, 4])
    dk, dv = k.cuda(), k.flip(1).contiguous().cuda()
    new = fa.fa512_cache_compact(dk, dv, table.cuda(), i32(lens).cuda(), acc.cuda(), n.cuda(), q_len=12, q_lens=i32(cnts).cuda())
    for got, src in ((dk, k), (dv, k.flip(1))):
        want, lens_want = paged.cache_compact(src.numpy(), table, i32(lens), acc, n, 12, i32(cnts))
        assert np.array_equal(got.cpu().numpy(), want)
    assert np.array_equal(new.cpu().numpy(), lens_want) and fa.fa512_device_status() == 0


def test_fork_copies_4_bit_pages(fa):
    psz, hk, layers, pool = 64, 2, 2, 16
    lens = [100, 64, 130]
    table = tables(lens, psz, 4, pool, 32, -1)
    refs = torch.zeros(pool, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    k = torch.from_numpy(np.random.RandomState(5).randint(0, 256, (layers, pool, psz, hk, ROW)).astype(np.uint8))
    parents = i32([2, 0, 2, 2, 1])
    dk, dv = k.cuda(), k.cuda()
    t, n, r = fa.fa512_cache_fork(dk, dv, table.cuda(), i32(lens).cuda(), parents.cuda(), refs.cuda())
    wk, _, wt, wn, wr = paged.cache_fork(k.numpy(), k.numpy(), table, i32(lens), parents, refs)
    assert np.array_equal(dk.cpu().numpy(), wk) and np.array_equal(dv.cpu().numpy(), wk)
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(n.cpu().numpy(), wn) and np.array_equal(r.cpu().numpy(), wr)
