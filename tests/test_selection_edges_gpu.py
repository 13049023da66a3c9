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


def list_call(fa, kind, rows, lens, lists, hk):
    """Attention over lists [batch][hk] of entries, padded with -1; pages of 16, in order."""
    width = max(1, max(paged.pages_of(n, 16) for n in lens))
    n_sel = max(len(x) for per in lists for x in per)
    sel = np.full((len(lens), hk, n_sel), -1, dtype=np.int32)
    for b, per in enumerate(lists):
        for h, x in enumerate(per):
            sel[b, h, :len(x)] = x
    table = torch.arange(len(lens) * width, dtype=torch.int32).view(len(lens), width)
    shape = (len(lens) * width, 16, hk)
    if kind == "bf16":
        call, k = fa.fa512_decode_paged_sparse, torch.ones(*shape, D, dtype=torch.bfloat16)
    elif kind == "e4m3":
        call, k = fa.fa512_decode_paged_sparse_fp8, torch.full((*shape, D), 0x38, dtype=torch.uint8)
    else:
        call, k = fa.fa512_decode_paged_sparse_fp4, torch.full((*shape, 288), 0x22, dtype=torch.uint8)
    q = workloads.draft_queries(len(lens), 1, rows * hk, seed=5)
    o, l = call(q.cuda(), k.cuda(), k.cuda(), table.cuda(), i32(lens).cuda(), torch.from_numpy(sel).cuda(),
                max_kv_len=width * 16)
    torch.cuda.synchronize()
    assert torch.isfinite(o).all()
    return l.view(len(lens), hk, rows).cpu()


KINDS = pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])


@KINDS
@pytest.mark.parametrize("rows", [2, 12])
def test_entries_behind_a_sequence_s_pages_are_recorded(fa, kind, rows):
    """A list may have more entries than its sequence has pages; those name none."""
    late = [[-1] * 54 + list(range(10)), list(range(10)) + [10], list(range(10)) + [3], [0, 1] + [-1] * 60 + [5],
            [-1] * 10 + [0], [9] + [-1] * 9 + [1 << 30]]
    every = list(range(10))
    l = list_call(fa, kind, rows, [160, 150, 0, 1], [[[9] + [-1] * 70, every], [[0, 3, 9], every], [[], []], [[0], []]], 2)
    assert fa.fa512_device_status() == 0
    assert torch.isneginf(l[2]).all()
    for bad in late:
        list_call(fa, kind, rows, [150], [[bad]], 1)
        assert fa.fa512_device_status() == 6, bad
        for b in range(3):                               # beside others, of the second KV head
            lists = [[list(range(4)), list(range(4))] for _ in range(3)]
            lists[b][1] = bad
            list_call(fa, kind, rows, [150, 160, 145], lists, 2)
            assert fa.fa512_device_status() == 6, (bad, b)
    for bad in ([0], [-1, 0], [-1] * 70 + [7]):           # no pages at all
        l = list_call(fa, kind, rows, [0, 150], [[bad], [[0, 1]]], 1)
        assert fa.fa512_device_status() == 6, bad
        assert torch.isneginf(l[0]).all()


@KINDS
@pytest.mark.parametrize("q_len,hq,hk", [(1, 8, 4), (1, 8, 1), (4, 8, 2), (2, 3, 1)])
@pytest.mark.parametrize("window", [0, 70])
def test_against_the_dense_call(fa, kind, q_len, hq, hk, window):
    """Lists of all pages against the dense call, and the dense 4-bit call under a window against the reference.

    Tolerance of each call's output, A = sum p |v| / sum p (fp64): 2^-8 |O| (bf16), 1e-3 A (the scores), 1e-6, and
    the weights' rounding: 2^-8 A to bf16 (dense E4M3 too, for the rows it widens to bf16), 2^-10 A to f16 with 2^-26 n
    vmax for those below its normal range.
    """
    lens, psz = [1000, 130, 64, q_len], 64
    need = [paged.pages_of(n, psz) for n in lens]
    table = np.zeros((len(lens), max(need)), dtype=np.int32)
    sel = np.full((len(lens), hk, max(need)), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = np.arange(at, at + k)[::-1]
        sel[b, :, :k] = np.arange(k)
        at += k
    rng = np.random.RandomState(9)
    x = [torch.tensor(rng.randn(at, psz, hk, D), dtype=torch.float32).to(torch.bfloat16) for _ in range(2)]
    kw, vmax = {}, float(x[1].float().abs().max())
    if kind == "e4m3":
        kw = {"k_scale": 0.0371, "v_scale": 0.0517}
        x = [(y.float() / s).to(torch.float8_e4m3fn).view(torch.uint8) for y, s in zip(x, (0.0371, 0.0517))]
    elif kind == "e2m1":
        kw = {"k_scale": 0.25, "v_scale": 1.3}
        x = [torch.from_numpy(paged.fp4_rows(y, s)) for y, s in zip(x, (0.25, 1.3))]
    table, n, sel = torch.from_numpy(table), i32(lens), torch.from_numpy(sel)
    q = workloads.draft_queries(len(lens), q_len, hq, seed=4)
    args = (q, x[0], x[1], table, n)
    dense, lists = {"bf16": (fa.fa512_decode_paged_q, fa.fa512_decode_paged_sparse),
                    "e4m3": (fa.fa512_decode_paged_fp8, fa.fa512_decode_paged_sparse_fp8),
                    "e2m1": (fa.fa512_decode_paged_fp4, fa.fa512_decode_paged_sparse_fp4)}[kind]
    on = [y.cuda() for y in args]
    ref, rl, weight = paged.decode_paged_any(*args, window=window, **kw)
    base = 2.0 ** -8 * np.abs(ref) + 1e-3 * weight + 1e-6
    f16 = 2.0 ** -10 * weight + 2.0 ** -26 * max(lens) * 1.5 * vmax
    bf16 = 2.0 ** -8 * weight
    of_dense, of_lists = base + (f16 if kind == "e2m1" else bf16), base + (bf16 if kind == "bf16" else f16)
    o, l = (y.float().cpu().numpy().astype(np.float64) for y in dense(*on, max_kv_len=1000, window=window, **kw))
    assert np.all(np.abs(o - ref) <= of_dense) and np.max(np.abs(l - rl)) <= 1e-3
    if not window:
        s, m = (y.float().cpu().numpy().astype(np.float64) for y in lists(*on, sel.cuda(), max_kv_len=1000, **kw))
        assert np.all(np.abs(s - ref) <= of_lists) and np.max(np.abs(m - rl)) <= 1e-3
        assert np.all(np.abs(s - o) <= of_dense + of_lists) and np.max(np.abs(m - l)) <= 1e-4
    assert fa.fa512_device_status() == 0
