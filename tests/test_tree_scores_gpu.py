"""Scores of any finite size: one key far above the others, at every place of a tile and in every tile."""
import numpy as np
import pytest
import torch

from head_dim_flashattention_gb300 import workloads
from oracle import paged
from test_decode_tree_gpu import FP8, call, compare, fa, make  # noqa: F401

pytestmark = pytest.mark.gpu
D = 512


@FP8
@pytest.mark.parametrize("q_len", [4, 20, 40])                    # 8, 40 and 80 rows of a KV head
@pytest.mark.parametrize("power", [10, 27, 33, 70, 110])
@pytest.mark.parametrize("splits", [1, 3])
def test_large_scores(fa, splits, power, q_len, fp8):             # noqa: F811
    """q is 2^power everywhere and the key of one position 1 everywhere, so its score is 2^power 512^1/2, several times
    any other's, and O that position's V.

    Its 512 products and their sums are exact; the LSE is off by the roundings of the scale, of log2 e, of their product
    with the score, of ln 2 and of its product, and of the output: 6 x 2^-24 of it, below 2^-21."""
    lens = [700, 700, 700, 700]
    pc, q, s = make(lens, q_len, 8, 4, 64, 151, fp8)
    one = workloads.to_e4m3(torch.ones(4, D), s["k_scale"]) if fp8 else torch.ones(4, D).to(torch.bfloat16)
    for b, pos in enumerate((5, 130, 300, 700 - q_len)):
        pc.k_pages[int(pc.page_table[b, pos // 64]), pos % 64] = one
    q = torch.full_like(q, 2.0 ** power)
    o, l = call(fa, pc, q, None, s, num_splits=splits)
    assert fa.fa512_device_status() == 0
    ro, rl, weight = paged.decode_paged_tree(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, None, **s)
    assert np.all(rl >= 2.0 ** power * 22)
    assert np.all(np.abs(l - rl) <= 2.0 ** -21 * rl)
    compare((o, rl), (ro, rl, weight))
