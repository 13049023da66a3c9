"""Selected pages at the edges: queries that are not numbers, lists with entries where no pages are."""
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


@pytest.mark.parametrize("q_len,hq,hk", [(1, 8, 4), (1, 1, 1), (1, 16, 1), (4, 8, 4), (3, 3, 1)])
@pytest.mark.parametrize("channel", [0, 7, 255, 256, 511])
def test_select_with_a_nan_in_a_query(fa, q_len, hq, hk, channel):
    """Every score of that (sequence, KV head) is NaN: equal ones, by their number; the others are chosen as ever."""
    psz, pick, lens = 16, 9, [1600, 1111, 2, 300]
    need = [paged.pages_of(n, psz) for n in lens]
    rng = np.random.RandomState(channel)
    table = np.zeros((len(lens), max(need)), dtype=np.int32)
    perm, at = rng.permutation(sum(need)), 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    table, n = torch.from_numpy(table), i32(lens)
    w = 2.0 + 0.6 * rng.rand(sum(need), hk, 2, D)
    w[:, :, 0] *= -1
    bounds = torch.tensor(w, dtype=torch.float32).to(torch.bfloat16)
    q = workloads.draft_queries(len(lens), q_len, hq, seed=3)
    q[0, q_len - 1, 0, channel] = float("nan")            # the first sequence's first KV head
    q[3, 0, hq - 1, channel] = float("nan")               # the last one's last
    if q_len > 2:
        q[2, 0, :, channel] = float("nan")                # before the third one's first position: not looked at
    got = fa.fa512_select_pages(q.cuda(), bounds.cuda(), table.cuda(), n.cuda(), page_size=psz, n_select=pick,
                                n_first=1, n_last=2).cpu().numpy()
    assert fa.fa512_device_status() == 0
    want = paged.select_pages(q, bounds, table, n, psz, pick, 1, 2)
    for b, h in ((0, 0), (3, hk - 1)):
        by_number = list(range(pick - 2)) + [need[b] - 2, need[b] - 1]
        assert want[b, h].tolist() == by_number and got[b, h].tolist() == by_number
    assert np.array_equal(got, want)
