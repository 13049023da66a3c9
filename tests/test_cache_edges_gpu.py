"""Counts, layers, pages and tables at the edges of what the cache calls take."""
import numpy as np
import pytest
import torch

from head_dim_flashattention_gb300 import workloads
from oracle import paged
from test_cache_gpu import FP8, bits, fa, i32, random_pages  # noqa: F401

pytestmark = pytest.mark.gpu
D = 512


@FP8
@pytest.mark.parametrize("count", [4, 1000, 2 ** 31 - 1, -1, -2 ** 31])
def test_append_writes_nothing_for_a_count_out_of_range(fa, count, fp8):   # noqa: F811
    """The other sequence's rows are written."""
    k = random_pages((4, 16, 2, D), fp8, 5)
    kn = workloads.randn_bf16((2, 3, 2, D), 97)
    pt, lens = i32([[0, 1], [2, 3]]), [10, 12]
    kc, vc = k.cuda(), k.cuda()
    f = fa.fa512_cache_append_fp8 if fp8 else fa.fa512_cache_append
    f(kn.cuda(), kn.cuda(), kc, vc, pt.cuda(), i32(lens).cuda(), q_lens=i32([count, 3]).cuda())
    assert fa.fa512_device_status() == 6
    want = paged.cache_append(kn, bits(k), pt, lens, i32([0, 3]), 1.0 if fp8 else None)
    assert np.array_equal(bits(kc), want) and np.array_equal(bits(vc), want)


def test_compact_of_a_cache_without_layers(fa):                    # noqa: F811
    k = torch.empty((0, 4, 16, 1, D), dtype=torch.bfloat16, device="cuda")
    args = (i32([[0, 1], [2, 3]]).cuda(), i32([20, 30]).cuda(), i32([[1, 2], [0, 3]]).cuda(), i32([2, 1]).cuda())
    new = fa.fa512_cache_compact(k, k, *args, q_len=8)
    assert new.tolist() == [14, 23] and fa.fa512_device_status() == 0


@FP8
@pytest.mark.parametrize("bad", [9, 4, -1, -2 ** 31])
def test_fork_of_a_partly_filled_page_that_is_none(fa, bad, fp8):  # noqa: F811
    """No child gets a page for it; the other parent's second child gets the lowest free one, and its rows."""
    k = random_pages((2, 4, 16, 1, D), fp8, 13)
    v = random_pages((2, 4, 16, 1, D), fp8, 14)
    kc, vc = k.cuda(), v.cuda()
    t, n, r = fa.fa512_cache_fork(kc, vc, i32([[3, bad], [0, -1]]).cuda(), i32([20, 3]).cuda(), i32([0, 0, 1, 1]).cuda(),
                                  i32([1, 0, 0, 1]).cuda())
    assert fa.fa512_device_status() == 6
    assert t.tolist() == [[3, -1], [3, -1], [0, -1], [1, -1]] and n.tolist() == [20, 20, 3, 3]
    assert r.tolist() == [1, 1, 0, 2]
    for got, was in ((bits(kc), bits(k)), (bits(vc), bits(v))):
        want = was.copy()
        want[:, 1, :3] = was[:, 0, :3]
        assert np.array_equal(got, want)


def test_compact_with_a_page_outside_the_pool(fa):                 # noqa: F811
    """The rows that lie in it stay, the others move, and the length is the usual one."""
    k = random_pages((2, 4, 16, 1, D), False, 15)
    kc, vc = k.cuda(), k.cuda()
    pt, lens = [[0, 77], [2, 3]], [20, 30]
    new = fa.fa512_cache_compact(kc, vc, i32(pt).cuda(), i32(lens).cuda(), i32([[1, 2, 7], [0, 2, 3]]).cuda(), i32([3, 3]).cuda(),
                                 q_len=8)
    assert fa.fa512_device_status() == 6 and new.tolist() == [15, 25]
    want, _ = paged.cache_compact(bits(k), i32([[0, 0], [2, 3]]), lens, [[1, 2, -1], [0, 2, 3]], [2, 3], 8)
    assert np.array_equal(bits(kc), want) and np.array_equal(bits(vc), want)


@FP8
def test_a_sequence_shortened_into_a_shared_page_grows_on_its_own(fa, fp8):    # noqa: F811
    """Two children share a whole page; one is cut back to inside it, forked into two, the first of them ended, and the
    second takes new rows: the sibling's rows are as they were, and the counts agree with the tables."""
    psz, pool, hk = 16, 12, 2
    k = random_pages((1, pool, psz, hk, D), fp8, 16).cuda()
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    table, refs = fa.fa512_cache_resize(torch.full((1, 4), -1, dtype=torch.int32, device="cuda"), i32([0]).cuda(),
                                        i32([40]).cuda(), refs, page_size=psz)
    table, lens, refs = fa.fa512_cache_fork(k, k, table, i32([40]).cuda(), i32([0, 0]).cuda(), refs)
    shorter = i32([21, 40]).cuda()                                 # inside the second page, which both hold
    table, refs = fa.fa512_cache_resize(table, lens, shorter, refs, page_size=psz)
    assert table[0, 1] == table[1, 1] and refs[table[0, 1]] == 2
    table, lens, refs = fa.fa512_cache_fork(k, k, table, shorter, i32([0, 0, 1]).cuda(), refs)
    grown = i32([0, 30, 40]).cuda()
    table, refs = fa.fa512_cache_resize(table, lens, grown, refs, page_size=psz)
    before = bits(k)
    assert table[1, 1] != table[2, 1]
    new = workloads.randn_bf16((3, 9, hk, D), 98).cuda()
    append = fa.fa512_cache_append_fp8 if fp8 else fa.fa512_cache_append
    append(new, new, k[0], k[0], table, grown, q_lens=i32([0, 9, 0]).cuda())
    t, after = table.cpu().numpy(), bits(k)
    for page in t[2, :3]:
        assert np.array_equal(after[0, page], before[0, page])
    mine = paged.cache_append(new.cpu(), before[0], t, [0, 30, 40], i32([0, 9, 0]), 1.0 if fp8 else None)
    assert np.array_equal(after[0], mine) and np.array_equal(after[0, t[1, 1], :5], before[0, t[2, 1], :5])
    assert np.array_equal(refs.cpu().numpy(), np.bincount(t[t >= 0], minlength=pool)) and fa.fa512_device_status() == 0
