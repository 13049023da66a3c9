"""The tree calls' workspace: bounded whatever the batch, and nothing behind its size is written."""
import numpy as np
import pytest
import torch

import __graft_entry__
import head_dim_flashattention_gb300 as fa
from test_decode_tree_gpu import FP8, call, check, make

D = 512


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    fa.load_library()


@pytest.mark.parametrize("shape", [(8, 4096, 32, 4, 16384), (15, 4096, 32, 4, 28672), (512, 1, 8, 4, 28672),
                                   (64, 64, 8, 4, 28672), (1, 65535, 128, 1, 65536), (16, 300, 128, 1, 131072)])
@pytest.mark.parametrize("splits", [0, 2, 1024])
def test_the_size_is_bounded(shape, splits):
    """64 MB of partials (above that two segments a CTA or pair: 152 x 2 x 64 rows of 512 floats and two, 40 MB), and 8
    bytes for each (sequence, row group, KV head)."""
    batch, q_len, hq, hk, _ = shape
    items = batch * -(-q_len * (hq // hk) // 32) * hk
    assert fa.fa512_decode_workspace_bytes_tree(*shape, 0, 0, splits) <= (64 << 20) + 8 * items + 3 * 256


@pytest.mark.parametrize("shape", [(2, 4, 516, 4, 200), (65536, 1, 8, 4, 200), (2, 1, 65536, 65536, 200),
                                   (2, 1 << 20, 8, 4, 1 << 21), (1, 2 ** 31 - 1, 128, 1, 200),
                                   (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1, 2 ** 31 - 1)])
def test_shapes_that_the_calls_refuse_have_no_size(shape):
    """And one split, whatever their products overflow to."""
    assert fa.fa512_decode_workspace_bytes_tree(*shape) == 0
    assert fa.fa512_decode_workspace_bytes_tree(*shape, 0, 0, 7) == 0
    assert fa.fa512_decode_auto_splits_tree(*shape) == 1
    assert fa.fa512_decode_auto_splits_tree(4, 16383, 8388480, 65535, 2 ** 31 - 1) == 1     # accepted by itself, not with as many keys


@pytest.mark.gpu
@FP8
@pytest.mark.parametrize("batch,q_len,hq,splits", [(50, 20, 8, 0), (30, 5, 8, 9), (3, 300, 8, 0), (4, 300, 8, 40), (5, 75, 32, 3),
                                                   (2, 4, 8, 5), (3, 3, 8, 1024), (2, 16, 8, 1024), (1, 70, 8, 1024), (1, 4, 8, 1024)])
def test_nothing_behind_it_is_written(batch, q_len, hq, splits, fp8):
    lens = [q_len + 37 * (i % 11) + 900 * (i % 3 == 0) for i in range(batch)]
    pc, q, s = make(lens, q_len, hq, 4, 64, 161, fp8)
    need = fa.fa512_decode_workspace_bytes_tree(batch, q_len, hq, 4, pc.max_kv_len, 0, 0, splits)
    buf = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    got = check(fa, pc, q, None, s, num_splits=splits, workspace=buf[4096:4096 + need])
    assert torch.all(buf[:4096] == 0x5A) and torch.all(buf[4096 + need:] == 0x5A)
    again = call(fa, pc, q, None, s, num_splits=splits)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [0, 1, 7])
def test_a_long_run_agrees_with_the_paged_prefill(splits):
    """Runs of 2,000 tokens and 8 heads a KV head, 5 of them ragged: 125 row groups each.

    Each call is off by 2^-8 |O| + (2^-8 + 1e-3) A (see test_decode_tree_gpu.py); with 1,000 keys and more A, the mean
    |v| of normal values, stays below 1."""
    lens, cnts = [3000, 4096, 3333, 3100, 3700], [2000, 2000, 1999, 700, 1]
    pc, q, _ = make(lens, 2000, 32, 4, 64, 162)
    ql = torch.tensor(cnts, dtype=torch.int32)
    o, l = call(fa, pc, q, None, {}, q_lens=ql, num_splits=splits)
    rows = torch.cat([q[b, :n] for b, n in enumerate(cnts)]).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(cnts)]), dtype=torch.int32).cuda()
    po, pl = fa.fa512_prefill_paged(rows, pc.k_pages.cuda(), pc.v_pages.cuda(), pc.page_table.cuda(), cu,
                                    pc.kv_lens.cuda(), max_seqlen_q=2000)
    po, pl = po.float().cpu().numpy(), pl.cpu().numpy()
    assert fa.fa512_device_status() == 0
    at = 0
    for b, n in enumerate(cnts):
        want, wl = po[at:at + n], pl[:, at:at + n].T
        at += n
        assert np.all(np.abs(o[b, :n] - want) <= 2.0 ** -7 * np.abs(want) + 2 * (2.0 ** -8 + 1e-3))
        assert np.max(np.abs(l[b, :n] - wl)) <= 2e-3
        assert np.all(o[b, n:] == 0) and np.all(np.isneginf(l[b, n:]))


def test_more_key_tiles_than_fit_are_refused():
    """2^15 sequences, 2^13 row groups, 2^15 KV heads and 2^21 tiles: 2^64 of them."""
    lib = fa.load_library()
    for tiles in (1 << 21, 1 << 20, 1):
        status = lib.fa512_decode_paged_tree(16, 16, 16, 16, 16, None, None, 16, None, 1 << 15, 1 << 13, 1 << 22, 1 << 15, 256, 4,
                                             1 << 21, tiles * 256, 0.05, 0, 0, 1, None, 0, None)
        assert status == 2, tiles
