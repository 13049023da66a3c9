"""Infinities and NaN that rows do see: the tree call's rows come out NaN where
the formula's do, and no other row does."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_decode_tree_gpu import FP8, call, compare, fa, make, random_masks  # noqa: F401

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def check_rows(fa, pc, q, mask, scales, huge=None, **kw):
    """NaN in the rows where the reference has it, the usual tolerance everywhere else.

    huge: a row whose LSE is of the order of 2^124, where an absolute 1e-3 is far below fp32's half step.  Its query
    holds 2^127 beside 508 elements up to 4.5 x 2^100, which the two E4M3 terms (steps of 2^-16 of the largest) drop:
    at most 508 x 4.5^2 x 2^100 < 2^114 of a score's 2^127 |k|, and the row's largest |k| there is above 2^-2; fp32's
    sums of 512 products stay below 2^-14.  In all 2^-11 of the LSE at most."""
    o, l = call(fa, pc, q, mask, scales, **kw)
    assert fa.fa512_device_status() == 0
    with np.errstate(invalid="ignore"):
        ro, rl, weight = paged.decode_paged_tree(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, mask, **scales)
    bad = np.isnan(rl)
    assert np.array_equal(bad, np.isnan(ro).all(-1)) and bad.any() and not bad.all()
    assert np.array_equal(np.isnan(l), bad)
    assert np.all(np.isnan(o[bad]))
    if huge is not None:
        assert abs(rl[huge]) > 2.0 ** 100 and abs(l[huge] - rl[huge]) <= 2.0 ** -11 * abs(rl[huge])
        l[huge] = rl[huge] = 0.0
    compare((o[~bad], l[~bad]), (ro[~bad], rl[~bad], weight[~bad]))


@pytest.mark.parametrize("hq", [8, 16, 32])                        # 18, 36 and 72 rows of a KV head
@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("fp8,bad", [(False, NAN), (False, INF), (False, -INF), (True, NAN)])
def test_queries(fa, fp8, bad, splits, hq):                        # noqa: F811
    pc, q, s = make([700, 90, 5, 128], 9, hq, 4, 64, 141, fp8)
    q[0, 3, 1, 77] = q[1, 0, hq - 1, 500] = q[3, 8, 0, 0] = bad
    check_rows(fa, pc, q, random_masks(4, 9, 141), s, num_splits=splits)


@FP8
@pytest.mark.parametrize("hq", [8, 256])                           # 2 and 64 rows; 128 of a pair are below
def test_the_only_key(fa, hq, fp8):                                # noqa: F811
    """A sequence's only key, one of a whole tile and one of a last partial tile."""
    pc, q, s = make([1, 300, 300, 300], 1, hq, 4, 64, 142, fp8)
    for b, pos in ((0, 0), (1, 40), (2, 299)):
        pc.k_pages[int(pc.page_table[b, pos // 64]), pos % 64] = 0x7F if fp8 else NAN
    check_rows(fa, pc, q, None, s)
    check_rows(fa, pc, q, None, s, num_splits=3)


@FP8
def test_a_drafted_key_that_some_rows_see(fa, fp8):                # noqa: F811
    """Only the rows whose mask names the token are NaN; 160 rows in two groups."""
    pc, q, s = make([20, 400], 20, 32, 4, 16, 143, fp8)
    mask = torch.zeros((2, 20, 1), dtype=torch.int32)
    for t in range(20):
        mask[:, t, 0] = 1 << t | (1 if t % 2 else 0)
    for b, n in ((0, 20), (1, 400)):
        pos = n - 20
        pc.k_pages[int(pc.page_table[b, pos // 16]), pos % 16] = 0x7F if fp8 else NAN
    check_rows(fa, pc, q, mask, s)


@pytest.mark.parametrize("hq", [8, 16, 32])
@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("bad", [INF, -INF])
def test_infinite_queries_over_fp8(fa, bad, splits, hq):           # noqa: F811
    """E4M3 has no infinity: the row's terms are NaN, not 448."""
    pc, q, s = make([700, 90, 5, 128], 9, hq, 4, 64, 144, True)
    q[0, 3, 1, 77] = q[1, 0, hq - 1, 500] = q[3, 8, 0, 0] = bad
    q[2, 4, 0, 3] = 2.0 ** 127                                     # the largest exponent of a finite value is one
    q[2, 4, 0, 4:] *= 2.0 ** 100
    check_rows(fa, pc, q, random_masks(4, 9, 144), s, huge=(2, 4, 0), num_splits=splits)
