"""Padded batches of the tree calls: what padding holds reaches nothing, padding's rows are written empty, and repeats
give the same bits."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_decode_tree_gpu import FP8, call, check, compare, fa, make, random_masks  # noqa: F401

pytestmark = pytest.mark.gpu


@FP8
@pytest.mark.parametrize("hq", [4, 8, 16])                        # 30, 60 and 120 rows of a KV head
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("splits", [0, 1])
def test_repeats_are_bitwise_equal_and_leave_padding_empty(fa, splits, tree, hq, fp8):   # noqa: F811
    lens, cnts = [1500, 700, 300, 40], [30, 0, 11, 1]
    pc, q, s = make(lens, 30, hq, 4, 64, 171, fp8)
    mask = random_masks(4, 30, 171) if tree else None
    for b, n in enumerate(cnts):
        q[b, n:] = float("nan")
        if tree:
            mask[b, n:] = -1
    ql = torch.tensor(cnts, dtype=torch.int32)
    runs = []
    for fill in (7.0, float("nan"), -3.0):
        out = torch.full(q.shape, fill, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:3], fill, dtype=torch.float32, device="cuda")
        runs.append(call(fa, pc, q, mask, s, q_lens=ql, out=out, lse=lse, num_splits=splits))
    for o, l in runs[1:]:
        assert np.array_equal(o, runs[0][0]) and np.array_equal(l, runs[0][1])
    for b, n in enumerate(cnts):
        assert np.all(runs[0][0][b, n:] == 0) and np.all(np.isneginf(runs[0][1][b, n:]))
    want = paged.decode_paged_tree(torch.nan_to_num(q), pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, mask, q_lens=ql, **s)
    compare(runs[0], want)
    assert fa.fa512_device_status() == 0


@FP8
@pytest.mark.parametrize("hq", [4, 16])
def test_nothing_to_see(fa, hq, fp8):                              # noqa: F811
    """No cached position at all: with the host's bound at 0 and above it; every row is written empty."""
    pc, q, s = make([64, 64], 20, hq, 4, 64, 172, fp8)
    pc.kv_lens[:] = 0
    for most in (0, 64):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        o, l = call(fa, pc, q, None, s, max_kv_len=most, out=out, window=5, n_sinks=2)
        assert np.all(o == 0) and np.all(np.isneginf(l)) and fa.fa512_device_status() == 0


@FP8
@pytest.mark.parametrize("hq", [4, 16])
def test_sinks_without_end(fa, hq, fp8):                           # noqa: F811
    """n_sinks at int32's end: the window hides nothing."""
    pc, q, s = make([900, 333], 20, hq, 4, 64, 173, fp8)
    a = check(fa, pc, q, None, s, window=50, n_sinks=2 ** 31 - 1)
    b = call(fa, pc, q, None, s)
    np.testing.assert_allclose(a[1], b[1], atol=1e-3)
