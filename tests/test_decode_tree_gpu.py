"""Parity of fa512_decode_paged_tree and its FP8 form (drafted tokens, a tree
or a plain run of any length, over a paged cache) with the fp64 reference.

Tolerance of an output element, with A = sum p |v| / sum p of its row (fp64):
  2^-8 |O|   the output's rounding to bf16 (half a step),
  2^-8 A     each p's rounding before P V (bf16, or three E5M2 terms: 2^-9),
  1e-3 A     the scores: products and sums in fp32; over an FP8 cache q is
             split into two E4M3 terms, off by at most 2^-18 of its row's
             largest element, so a score of 512 products with |q| <= 4.5,
             |k| <= 4.5 and scale 512^-1/2 is off by less than 4e-4 for random
             signs at 5 sigma, and p by that fraction,
plus 1e-6.  LSE: 1e-3 (as everywhere in these tests).
"""
import numpy as np
import pytest
import torch

from head_dim_flashattention_gb300 import workloads
from oracle import paged

pytestmark = pytest.mark.gpu
D = 512
NAN8 = 0x7F


@pytest.fixture(scope="module")
def fa(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    import head_dim_flashattention_gb300 as fa
    fa.load_library()
    return fa


def random_masks(batch, nodes, seed):
    """Random trees: node i sees itself and what its parent (an earlier node, or none) sees."""
    rng = np.random.RandomState(seed)
    words = np.zeros((batch, nodes, -(-nodes // 32)), dtype=np.int64)
    for b in range(batch):
        for i in range(nodes):
            up = rng.randint(-1, i) if i else -1
            if up >= 0:
                words[b, i] |= words[b, up]
            words[b, i, i // 32] |= 1 << (i % 32)
    return torch.from_numpy(words.astype(np.uint32).view(np.int32))


def make(lens, q_len, hq, hk, page, seed, fp8=False, poison=True):
    if fp8:
        pc, ks, vs = workloads.paged_fp8_inputs(len(lens), lens, hq, hk, page, seed=seed, poison=poison)
        scales = {"k_scale": ks, "v_scale": vs}
    else:
        pc = workloads.paged_decode_inputs(len(lens), lens, hq, hk, page, seed=seed, poison=poison)
        scales = {}
    return pc, workloads.draft_queries(len(lens), q_len, hq, seed=seed), scales


def poison_unseen(pc, mask, cnts, window, n_sinks):
    """NaN in every cached slot that no row sees; entries of pages nobody sees at all point outside the pool."""
    psz = pc.k_pages.shape[1]
    bad = NAN8 if pc.k_pages.dtype == torch.uint8 else float("nan")
    for b in range(len(cnts)):
        n = int(pc.kv_lens[b])
        seen = paged.tree_visible(mask, b, n, cnts[b], window, n_sinks).any(axis=0)
        for lp in range(-(-n // psz)):
            part = seen[lp * psz:(lp + 1) * psz]
            page = int(pc.page_table[b, lp])
            slots = torch.from_numpy(np.nonzero(~part)[0])
            pc.k_pages[page, slots] = bad
            pc.v_pages[page, slots] = bad


def call(fa, pc, q, mask, scales, dev="cuda", **kw):
    f = fa.fa512_decode_paged_tree_fp8 if scales else fa.fa512_decode_paged_tree
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    kw = {k: up(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    out, lse = f(up(q), up(pc.k_pages), up(pc.v_pages), up(pc.page_table), up(pc.kv_lens), up(mask),
                 **{"max_kv_len": pc.max_kv_len, **kw}, **scales)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def compare(got, want):
    (o, l), (ro, rl, weight) = got, want
    assert np.all(np.isfinite(o))
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 1e-3) * weight + 1e-6
    worst = np.max((np.abs(o - ro) - tol)) if o.size else 0.0
    assert worst <= 0, (worst, np.unravel_index(np.argmax(np.abs(o - ro) - tol), o.shape))
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(l), none)
    assert np.all(o[none] == 0)
    assert np.max(np.abs(l[~none] - rl[~none]), initial=0.0) <= 1e-3


def check(fa, pc, q, mask, scales, window=0, n_sinks=0, q_lens=None, **kw):
    got = call(fa, pc, q, mask, scales, window=window, n_sinks=n_sinks, q_lens=q_lens, **kw)
    assert fa.fa512_device_status() == 0
    want = paged.decode_paged_tree(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, mask, q_lens=q_lens,
                                   window=window, n_sinks=n_sinks, **scales)
    compare(got, want)
    return got


FP8 = pytest.mark.parametrize("fp8", [False, True])


@FP8
@pytest.mark.parametrize("nodes", [1, 2, 7, 31, 32, 33, 64, 65])
def test_tree_sizes(fa, nodes, fp8):
    lens = [nodes, nodes + 1, 700, 1153]
    pc, q, s = make(lens, nodes, 8, 4, 64, 71, fp8)
    check(fa, pc, q, random_masks(4, nodes, nodes), s)


@FP8
@pytest.mark.parametrize("nodes", [128, 256])
def test_large_trees(fa, nodes, fp8):
    pc, q, s = make([nodes + 130, 1000], nodes, 8, 4, 64, 72, fp8)
    check(fa, pc, q, random_masks(2, nodes, nodes), s)


@FP8
@pytest.mark.parametrize("hq,hk", [(32, 4), (16, 1), (12, 4), (4, 4), (1, 1), (80, 1), (128, 1)])
def test_head_groupings(fa, hq, hk, fp8):
    pc, q, s = make([300, 45], 9, hq, hk, 64, 73, fp8)
    check(fa, pc, q, random_masks(2, 9, 73), s)


@FP8
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(fa, page, fp8):
    pc, q, s = make([9, 127, 128, 129, 641], 9, 8, 4, page, 74, fp8)
    check(fa, pc, q, random_masks(5, 9, 74), s)
    check(fa, pc, q, None, s)


@FP8
@pytest.mark.parametrize("splits", [1, 2, 3, 16, 1024])
def test_split_invariance(fa, splits, fp8):
    pc, q, s = make([1000, 64, 4097], 10, 8, 4, 64, 75, fp8)
    check(fa, pc, q, random_masks(3, 10, 75), s, num_splits=splits)
    check(fa, pc, q, None, s, window=500, n_sinks=130, num_splits=splits)


@FP8
@pytest.mark.parametrize("q_len", [1, 5, 33, 150, 300])
def test_runs_of_tokens(fa, q_len, fp8):
    """No mask: a decode step, a few drafts, a chunk of several row tiles; caches shorter than the run too."""
    pc, q, s = make([q_len, q_len + 1, 517, 3], q_len, 8, 4, 64, 76, fp8)
    check(fa, pc, q, None, s)


@FP8
@pytest.mark.parametrize("window,n_sinks", [(1, 0), (1, 1), (5, 4), (64, 0), (128, 4), (130, 127), (200, 128),
                                            (200, 300), (5000, 4)])
@pytest.mark.parametrize("tree", [False, True])
def test_windows_and_sinks(fa, window, n_sinks, tree, fp8):
    """Slots that no row sees hold NaN."""
    lens = [12, 333, 1200, 2049]
    pc, q, s = make(lens, 12, 8, 4, 32, 77, fp8)
    mask = random_masks(4, 12, 77) if tree else None
    poison_unseen(pc, mask, [12] * 4, window, n_sinks)
    check(fa, pc, q, mask, s, window=window, n_sinks=n_sinks)
    check(fa, pc, q, mask, s, window=window, n_sinks=n_sinks, num_splits=3)


@FP8
def test_a_window_over_a_long_chunk(fa, fp8):
    pc, q, s = make([900, 470], 400, 16, 2, 64, 78, fp8)
    check(fa, pc, q, None, s, window=100, n_sinks=3)


@FP8
def test_padded_batches(fa, fp8):
    """q_lens of 0, of all and between; rows behind it are empty."""
    lens, cnts = [500, 41, 300, 13, 0], [17, 0, 20, 13, 0]
    pc, q, s = make(lens, 20, 8, 4, 64, 79, fp8)
    mask = random_masks(5, 20, 79)
    ql = torch.tensor(cnts, dtype=torch.int32)
    o, l = check(fa, pc, q, mask, s, q_lens=ql)
    assert np.all(o[1] == 0) and np.all(np.isneginf(l[1])) and np.all(np.isneginf(l[0, 17:]))
    check(fa, pc, q, None, s, q_lens=ql, window=30, n_sinks=2)


@FP8
def test_masks_that_leave_rows_empty(fa, fp8):
    """A token that sees no token sees the positions before the tree; where there are none, nothing."""
    pc, q, s = make([8, 200], 8, 8, 4, 64, 80, fp8)
    mask = random_masks(2, 8, 80)
    mask[:, 2] = 0
    mask[:, 7] = 0
    o, l = check(fa, pc, q, mask, s)
    assert np.all(np.isneginf(l[0, 2])) and np.all(np.isfinite(l[1, 2]))
    # bits at and behind q_lens[b] name tokens that are not there
    mask[:, 0] = -1
    check(fa, pc, q, mask, s, q_lens=torch.tensor([5, 6], dtype=torch.int32))


@FP8
def test_large_scores_keep_their_tail(fa, fp8):
    """One key far above thousands of others: their mass must survive the running maximum."""
    pc, q, s = make([4000, 4000], 4, 8, 4, 64, 81, fp8, poison=False)
    page, slot = int(pc.page_table[0, 5]), 9
    if fp8:
        pc.k_pages[page, slot] = workloads.to_e4m3(torch.full((4, D), 0.5), s["k_scale"])
    else:
        pc.k_pages[page, slot] = 0.5
    q[0] = 0.75          # score of that key: 512 * 0.375 / sqrt(512) = 8.5
    check(fa, pc, q, None, s)
    check(fa, pc, q, None, s, scale=None, num_splits=4)


@FP8
@pytest.mark.parametrize("scale", [0.0, -0.04, 0.3])
def test_scales(fa, scale, fp8):
    """scale 0 weighs all keys alike, a negative one turns the order round."""
    pc, q, s = make([300, 90], 6, 8, 4, 64, 82, fp8)
    mask = random_masks(2, 6, 82)
    got = call(fa, pc, q, mask, s, scale=scale)
    want = paged.decode_paged_tree(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, mask, scale=scale, **s)
    if scale == 0.3:     # scores 7 times the usual: their errors too (see the head of the file)
        o, l = got
        tol = 2.0 ** -8 * np.abs(want[0]) + (2.0 ** -8 + 7e-3) * want[2] + 1e-6
        assert np.all(np.abs(o - want[0]) <= tol) and np.max(np.abs(l - want[1])) <= 7e-3
    else:
        compare(got, want)


def test_extreme_queries_over_fp8(fa):
    """Rows of q far outside the range of E4M3 are scaled, not clipped."""
    pc, q, s = make([260, 70], 4, 8, 4, 64, 83, True)
    q = q * torch.tensor([2.0 ** 20, 2.0 ** -30, 1.0, 2.0 ** -100]).view(1, 4, 1, 1)
    q = q.to(torch.bfloat16)
    got = call(fa, pc, q, None, s, scale=512 ** -0.5 * 2.0 ** -20)
    want = paged.decode_paged_tree(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, None,
                                   scale=512 ** -0.5 * 2.0 ** -20, **s)
    compare(got, want)


def test_agrees_with_the_causal_decode(fa):
    """Without a mask it is fa512_decode_paged_q, which other kernels compute."""
    pc, q, _ = make([900, 64, 130], 4, 8, 4, 64, 84)
    o, l = call(fa, pc, q, None, {})
    a, b = fa.fa512_decode_paged_q(q.cuda(), pc.k_pages.cuda(), pc.v_pages.cuda(), pc.page_table.cuda(),
                                   pc.kv_lens.cuda(), max_kv_len=pc.max_kv_len)
    torch.cuda.synchronize()
    np.testing.assert_allclose(o, a.float().cpu().numpy(), atol=1e-2)
    np.testing.assert_allclose(l, b.cpu().numpy(), atol=1e-3)


@FP8
def test_repeats_are_bitwise_equal_and_leave_padding_alone(fa, fp8):
    pc, q, s = make([1500, 700], 30, 8, 4, 64, 85, fp8)
    mask = random_masks(2, 30, 85)
    a = call(fa, pc, q, mask, s)
    b = call(fa, pc, q, mask, s)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@FP8
def test_many_tiles_of_edges_repeat_bitwise(fa, fp8):
    """Bands that start and end inside tiles, in more blocks than fit the GPU at once: every run gives the same bits."""
    lens = [4000 - 37 * i for i in range(8)]
    pc, q, s = make(lens, 75, 32, 4, 64, 90, fp8)
    args = dict(window=1000, n_sinks=4)
    a = check(fa, pc, q, None, s, **args)
    for _ in range(4):
        b = call(fa, pc, q, None, s, **args)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_outputs_may_sit_inside_larger_buffers(fa):
    """Bytes before and behind out and lse keep what they held."""
    pc, q, s = make([300, 90], 7, 8, 4, 64, 86)
    n = q.numel()
    buf = torch.full((n + 1024,), 7.0, dtype=torch.bfloat16, device="cuda")
    lbuf = torch.full((2 * 7 * 8 + 64,), 7.0, dtype=torch.float32, device="cuda")
    out, lse = buf[512:512 + n].view(q.shape), lbuf[32:32 + 112].view(2, 7, 8)
    call(fa, pc, q, None, s, out=out, lse=lse)
    assert torch.all(buf[:512] == 7) and torch.all(buf[512 + n:] == 7)
    assert torch.all(lbuf[:32] == 7) and torch.all(lbuf[-32:] == 7)


def test_no_lse_and_other_stream(fa):
    pc, q, _ = make([300, 90], 7, 8, 4, 64, 87)
    args = [t.cuda() for t in (q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens)]
    want, _ = fa.fa512_decode_paged_tree(*args, max_kv_len=300)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, none = fa.fa512_decode_paged_tree(*args, max_kv_len=300, return_lse=False, stream=side)
    side.synchronize()
    assert none is None and torch.equal(got, want)


def test_captured_and_replayed_with_new_lengths(fa):
    """A captured call follows the lengths, tables and queries that the buffers hold at each replay."""
    pc, q, _ = make([900, 700], 8, 8, 4, 64, 88)
    mask = random_masks(2, 8, 88).cuda()
    args = [t.cuda() for t in (q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens)]
    ws = torch.empty(fa.fa512_decode_workspace_bytes_tree(2, 8, 8, 4, 900), dtype=torch.uint8, device="cuda")
    fa.fa512_decode_paged_tree(*args, mask, max_kv_len=900, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = fa.fa512_decode_paged_tree(*args, mask, max_kv_len=900, workspace=ws)
    for lens in ([900, 700], [8, 333], [129, 0]):
        args[4].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        pc.kv_lens = torch.tensor(lens, dtype=torch.int32)
        want = paged.decode_paged_tree(q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens, mask.cpu())
        compare((out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)), want)


@FP8
def test_bad_pages_and_lengths_are_reported_not_read(fa, fp8):
    pc, q, s = make([200, 100], 5, 8, 4, 64, 89, fp8)
    good = pc.page_table.clone()
    pc.page_table[1, 0] = 10 ** 6
    call(fa, pc, q, None, s)
    assert fa.fa512_device_status() == 6 and fa.fa512_device_status() == 0
    pc.page_table[1, 0] = -5
    call(fa, pc, q, None, s)
    assert fa.fa512_device_status() == 6
    pc.page_table = good
    call(fa, pc, q, None, s, max_kv_len=150)
    assert fa.fa512_device_status() == 6
    call(fa, pc, q, None, s, q_lens=torch.tensor([6, 5], dtype=torch.int32))
    assert fa.fa512_device_status() == 6
    call(fa, pc, q, None, s, q_lens=torch.tensor([-1, 5], dtype=torch.int32))
    assert fa.fa512_device_status() == 6
    check(fa, pc, q, None, s)


@FP8
@pytest.mark.parametrize("window,n_sinks", [(1, 1), (5, 4), (200, 128), (200, 300), (700, 0), (5000, 4)])
@pytest.mark.parametrize("tree", [False, True])
def test_windows_and_sinks_of_many_rows(fa, window, n_sinks, tree, fp8):
    """Several row groups of one KV head; slots that no row sees hold NaN."""
    lens = [75, 333, 1200, 2049]
    pc, q, s = make(lens, 75, 8, 2, 32, 91, fp8)
    mask = random_masks(4, 75, 91) if tree else None
    poison_unseen(pc, mask, [75] * 4, window, n_sinks)
    check(fa, pc, q, mask, s, window=window, n_sinks=n_sinks)
    check(fa, pc, q, mask, s, window=window, n_sinks=n_sinks, num_splits=1)


@FP8
@pytest.mark.parametrize("hq", [4, 8, 16])
@pytest.mark.parametrize("window", [0, 3, 2 ** 31 - 1])
def test_trees_longer_than_the_cache(fa, window, hq, fp8):
    """Tokens whose position would be negative are not there; 32, 64 or 128 rows of a KV head."""
    lens, cnts = [20, 3, 0, 21, 90], [32, 30, 32, 21, 0]
    pc, q, s = make(lens, 32, hq, 4, 16, 92, fp8)
    ql = torch.tensor(cnts, dtype=torch.int32)
    mask = random_masks(5, 32, 92)
    mask[3, 5] = 0
    check(fa, pc, q, mask, s, window=window, q_lens=ql)
    check(fa, pc, q, mask, s, window=window, n_sinks=2, q_lens=ql)
    check(fa, pc, q, None, s, window=window, n_sinks=2, q_lens=ql)


@FP8
@pytest.mark.parametrize("nodes", [1, 20, 70])
@pytest.mark.parametrize("splits", [2, 32, 33, 60])
def test_each_way_of_merging(fa, splits, nodes, fp8):
    """Few rows or many, few segments or many; one sequence has none."""
    pc, q, s = make([9000, 0], nodes, 4, 2, 64, 93, fp8)
    pc.kv_lens[1] = 0
    check(fa, pc, q, None, s, num_splits=splits, q_lens=torch.tensor([nodes, 0], dtype=torch.int32))


@FP8
def test_sequences_may_share_pages(fa, fp8):
    """Two sequences over the same pages, a third with one page at several places."""
    pc, q, s = make([300, 300, 256], 40, 8, 4, 64, 94, fp8)
    pc.page_table[1] = pc.page_table[0]
    pc.page_table[2, 1:4] = pc.page_table[2, 0]
    q[1] = q[0]
    o, l = check(fa, pc, q, None, s)
    assert np.array_equal(o[0], o[1]) and np.array_equal(l[0], l[1])


@FP8
def test_pages_far_into_a_large_pool(fa, fp8):
    """Byte and element offsets past 32 bits: the same bits as over a small pool."""
    far, n, psz, hk = (34000 if fp8 else 17000), 25, 64, 4
    pc, q, s = make([700, 333], 33, 8, hk, psz, 95, fp8, poison=False)
    used = pc.k_pages.shape[0]
    assert used <= n and far * psz * hk * D > 2 ** 32 // (1 if fp8 else 2)
    big = [torch.empty((far + n,) + tuple(pc.k_pages.shape[1:]), dtype=pc.k_pages.dtype, device="cuda") for _ in range(2)]
    big[0][far:far + used].copy_(pc.k_pages)
    big[1][far:far + used].copy_(pc.v_pages)
    want = call(fa, pc, q, None, s)
    f = fa.fa512_decode_paged_tree_fp8 if fp8 else fa.fa512_decode_paged_tree
    o, l = f(q.cuda(), *big, (pc.page_table + far).cuda(), pc.kv_lens.cuda(), max_kv_len=pc.max_kv_len, **s)
    assert np.array_equal(o.float().cpu().numpy().astype(np.float64), want[0])
    assert np.array_equal(l.cpu().numpy().astype(np.float64), want[1])
    assert fa.fa512_device_status() == 0


def test_two_streams_at_once(fa):
    """Calls on two streams, of different shapes and each with its own workspace, give what they give alone."""
    jobs = []
    for nodes, seed in ((40, 96), (7, 97)):
        pc, q, _ = make([3000, 1500, 77], nodes, 8, 4, 64, seed)
        args = [t.cuda() for t in (q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens)]
        ws = torch.empty(fa.fa512_decode_workspace_bytes_tree(3, nodes, 8, 4, 3000), dtype=torch.uint8, device="cuda")
        want = [t.clone() for t in fa.fa512_decode_paged_tree(*args, max_kv_len=3000, workspace=ws)]
        jobs.append((args, ws, want, torch.cuda.Stream(), [torch.empty_like(t) for t in want]))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, ws, _, st, got in jobs:
            fa.fa512_decode_paged_tree(*args, None, *got, max_kv_len=3000, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for _, _, want, _, got in jobs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_graphs_share_a_workspace(fa):
    """Captured calls of different shapes over one workspace, replayed by turns on one stream."""
    ws = torch.empty(max(fa.fa512_decode_workspace_bytes_tree(2, n, 8, 4, 2000) for n in (33, 6)), dtype=torch.uint8,
                     device="cuda")
    graphs = []
    for nodes in (33, 6):
        pc, q, _ = make([2000, 900], nodes, 8, 4, 64, 98 + nodes)
        args = [t.cuda() for t in (q, pc.k_pages, pc.v_pages, pc.page_table, pc.kv_lens)]
        want = fa.fa512_decode_paged_tree(*args, max_kv_len=2000)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = fa.fa512_decode_paged_tree(*args, max_kv_len=2000, workspace=ws)
        graphs.append((g, got, want, args))
    for _ in range(3):
        for _, got, _, _ in graphs:
            got[0].fill_(9)
        for g, _, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, got, want, _ in graphs:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@FP8
@pytest.mark.parametrize("cnts", [[300, 300, 300, 300], [300, 290, 295, 300], [300, 1, 0, 17], [0, 0, 0, 40]])
def test_row_groups_of_padded_batches(fa, cnts, fp8):
    """Alike and unlike numbers of row groups in a batch: the work is dealt out differently."""
    pc, q, s = make([900, 300, 512, 777], 300, 8, 2, 64, 131, fp8)
    ql = torch.tensor(cnts, dtype=torch.int32)
    check(fa, pc, q, None, s, q_lens=ql)
    check(fa, pc, q, None, s, q_lens=ql, window=200, n_sinks=5, num_splits=1)
    check(fa, pc, q, None, s, q_lens=ql, window=600, num_splits=4)


@FP8
@pytest.mark.parametrize("hq", [8, 40])
@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("window,n_sinks", [(40, 3), (300, 70), (129, 128), (400, 260)])
def test_sinks_beside_a_window(fa, window, n_sinks, page, hq, fp8):
    """The keys between the sinks and the window are left out page by page; what no row sees holds NaN."""
    lens = [1100, 700, 271]
    pc, q, s = make(lens, 9, hq, 4, page, 132, fp8)
    mask = random_masks(3, 9, 132)
    poison_unseen(pc, mask, [9] * 3, window, n_sinks)
    check(fa, pc, q, mask, s, window=window, n_sinks=n_sinks)
    pc, q, s = make(lens, 9, hq, 4, page, 133, fp8)
    poison_unseen(pc, None, [9] * 3, window, n_sinks)
    check(fa, pc, q, None, s, window=window, n_sinks=n_sinks)


@FP8
@pytest.mark.parametrize("nodes", [3, 20, 40])
@pytest.mark.parametrize("shape", ["one long", "many"])
def test_ranges_over_several_items(fa, shape, nodes, fp8):
    """Lengths so unlike, or sequences so many, that a CTA's keys begin and end inside items of several sequences."""
    lens = [9000, 100, 90, 0, 700] if shape == "one long" else [60 + 37 * (i % 11) for i in range(50)]
    pc, q, s = make(lens, nodes, 8, 4, 64, 134, fp8)
    a = check(fa, pc, q, None, s)
    b = call(fa, pc, q, None, s)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    check(fa, pc, q, random_masks(len(lens), nodes, 134), s, num_splits=5)
    check(fa, pc, q, None, s, window=300, n_sinks=20)
