"""One key that takes most of the weight and whose value is 0 in the columns looked at,
beside thousands that share the rest (attention sinks): what those add up to must not
depend on the group scales of their values, on the rows of a KV head, nor on where
their reference lies against the row's.

Tolerance of an output element of column d, with A = sum p |v| / sum p (fp64):
  2^-8 |O|            the output's rounding to bf16 (half a step),
  (2^-10 + 1e-3) A    a weight's rounding to f16 and that of its product with the factor
                      between two references (half a step each); the scores in fp32,
  2^-26 n vmax_d      weights below f16's normal range: each of the two roundings is off
                      by at most 2^-25, and the largest weight is above 2^2,
plus 1e-7.  LSE: 1e-3.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged

pytestmark = pytest.mark.gpu
D, ROW, PSZ = 512, 288, 64


@pytest.fixture(scope="module")
def fa(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    import head_dim_flashattention_gb300 as fa
    fa.load_library()
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def fp4(values, scale_bytes):
    """[n, 512] values that are E2M1 values, [n, 32] scale bytes -> rows [n, 288]."""
    code = np.searchsorted(paged.E2M1, np.abs(values)).astype(np.uint8)
    assert np.array_equal(paged.E2M1[code], np.abs(values))
    code |= np.signbit(values).astype(np.uint8) << 3
    return np.concatenate([code[:, ::2] | (code[:, 1::2] << 4), scale_bytes.astype(np.uint8)], axis=1)


def cache(rows):
    """Rows of one sequence, one KV head -> pages, in order."""
    n = len(rows)
    pages = paged.pages_of(n, PSZ)
    out = np.zeros((pages * PSZ, 1, rows.shape[1]), dtype=rows.dtype)
    out[:n, 0] = rows
    return torch.from_numpy(out.reshape(pages, PSZ, 1, -1))


def run(fa, kind, sparse, q, k, v, n, scale, **kw):
    pages = k.shape[0]
    table, lens = torch.arange(pages, dtype=torch.int32)[None], i32([n])
    head = [q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda()]
    kw = {"max_kv_len": n, "scale": scale, **kw}
    if sparse:
        head.append(torch.arange(pages, dtype=torch.int32)[None, None].cuda())
        call = fa.fa512_decode_paged_sparse_fp8 if kind == "e4m3" else fa.fa512_decode_paged_sparse_fp4
    else:
        call = fa.fa512_decode_paged_fp4
    o, l = call(*head, **kw)
    torch.cuda.synchronize()
    assert fa.fa512_device_status() == 0
    return o.float().cpu().numpy().astype(np.float64), l.cpu().numpy().astype(np.float64), table, lens


def check(fa, kind, sparse, q, k, v, n, scale, **kw):
    o, l, table, lens = run(fa, kind, sparse, q, k, v, n, scale, **kw)
    ro, rl, weight = paged.decode_paged_any(q[:, None], k, v, table, lens, scale=scale)
    vmax = np.abs(paged.widen_cache(v)).reshape(-1, D).max(axis=0)
    err = np.abs(o - ro[:, 0])
    tol = 2.0 ** -8 * np.abs(ro[:, 0]) + (2.0 ** -10 + 1e-3) * weight[:, 0] + 2.0 ** -26 * n * vmax + 1e-7
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert np.all(err <= tol), (worst, o[worst], ro[:, 0][worst], tol[worst])
    assert np.max(np.abs(l - rl[:, 0])) <= 1e-3


@pytest.mark.parametrize("sparse,splits", [(False, 0), (False, 1), (True, 0), (True, 1)])
@pytest.mark.parametrize("rows", [1, 2, 3, 8, 16])
@pytest.mark.parametrize("n,rest", [(28672, 0.02), (28672, 0.05), (3000, 0.01), (700, 0.3)])
def test_small_group_scales_under_a_dominating_key(fa, n, rest, rows, sparse, splits):
    rng = np.random.RandomState(n + rows)
    k_values, v_values = np.zeros((n, D)), np.zeros((n, D))
    k_values[0, :16] = 6                                  # q k: 96 for the first key, 0 for the others
    v_values[1:] = 3 * np.sign(rng.randn(D))              # a column's values add up
    v_values[0, 1::2] = 6                                 # beside zeros in the even columns
    v_scales = np.broadcast_to(1 + np.arange(32) % 8, (n, 32)).copy()     # 2^-9 .. 2^-6
    v_scales[:, 24:] = rng.randint(1, 0x48, (n, 8))       # some groups' of all sizes, up to 3.75
    v_scales[0] = 0x50                                    # the first key's: 8
    k, v = cache(fp4(k_values, np.full((n, 32), 0x38))), cache(fp4(v_values, v_scales))
    q = torch.zeros(1, rows, D)
    q[..., :16] = 1
    score = math.log((n - 1) * (1 - rest) / rest)         # the others have `rest` of the weight together
    check(fa, "e2m1", sparse, q.to(torch.bfloat16), k, v, n, score / 96, num_splits=splits)


def sums(x):
    """[n] multiples of 0.5 up to 96 in size -> [n, 512] E2M1 values whose first 16 add up to them."""
    out, left = np.zeros((len(x), D)), np.abs(np.asarray(x, dtype=np.float64))
    for j in range(16):
        out[:, j] = paged.E2M1[np.searchsorted(paged.E2M1, np.minimum(left, 6), side="right") - 1]
        left -= out[:, j]
    assert not left.any()
    return out * np.sign(x)[:, None]


def stored(kind, values, scale_byte):
    """Rows of a cache that stand for ``values`` times the scale (4 bits) or for ``values`` (E4M3)."""
    if kind == "e2m1":
        return cache(fp4(values, np.full((len(values), 32), scale_byte)))
    return cache(torch.tensor(values, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


KINDS = pytest.mark.parametrize("kind,sparse", [("e2m1", False), ("e2m1", True), ("e4m3", True)])


@KINDS
@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("rows", [1, 2, 3, 8, 16])
@pytest.mark.parametrize("first,later", [(-24.5, -20.5), (-25.5, -21.5), (-30.5, -22.5), (-20.5, -20.5)])
def test_weights_far_below_another_block_s(fa, first, later, rows, splits, kind, sparse):
    """A dominating key in one block, all others in blocks whose reference, taken from lower scores than most of
    theirs, is 25 binades or more below."""
    n = 20000
    score = np.full(n, later)                             # log2 of the weights
    score[0], score[1:16], score[16:64] = 0.5, -60, first
    values = np.broadcast_to(3 * np.sign(np.random.RandomState(rows).randn(D)), (n, D)).copy()
    values[0] = 0
    q = torch.zeros(1, rows, D)
    q[..., :16] = 1
    check(fa, kind, sparse, q.to(torch.bfloat16), stored(kind, sums(score), 0x38), stored(kind, values, 0x38), n,
          math.log(2), num_splits=splits)


@KINDS
@pytest.mark.parametrize("rows", [1, 2, 3, 16])
@pytest.mark.parametrize("e", [22, 23, 24, 25, 26, 27, 28, 30])
def test_scores_a_step_of_fp32_apart(fa, e, rows, kind, sparse):
    """Scores near 2^e in log2 units, rising by one step of fp32 from block to block: no weight passes f16.  All
    values of a column are the same, and so is the output, within half a step of its bf16 and the weights' 2^-10."""
    n = 1500
    step = np.minimum(np.arange(n) // 16, 90).astype(np.float64)
    k_values = sums(np.full(n, 64.0))
    k_values[:, 16:32] = sums(step)[:, :16]
    top = 2688 if kind == "e2m1" else 448                 # the largest that the format holds
    sign = np.sign(np.random.RandomState(rows).randn(D))
    values = np.broadcast_to((6 if kind == "e2m1" else 448) * sign, (n, D))
    q = torch.zeros(1, rows, D)
    q[..., :16], q[..., 16:32] = 2.0 ** (e - 6), 2.0 ** (e - 23)
    for splits in (0, 1):
        o, l, _, _ = run(fa, kind, sparse, q.to(torch.bfloat16), stored(kind, k_values, 0x38),
                         stored(kind, values, 0x7E), n, math.log(2), num_splits=splits)
        assert np.max(np.abs(o - top * sign)) <= (2.0 ** -8 + 2.0 ** -10) * top
        assert np.all(np.abs(l / (2.0 ** e * math.log(2)) - 1) <= 2.0 ** -15)


@KINDS
@pytest.mark.parametrize("size", [1, 64])
@pytest.mark.parametrize("rows", [2, 3, 16])
def test_tensor_scales_next_to_the_smallest_float(fa, rows, size, kind, sparse):
    """A v_scale that is no normal float.  The tolerance of an ordinary one, times this one; beside it a step of 2^-149
    in each product and sum of a partial, and half a step of the output: bf16's smallest is 2^-133, and the outputs, up
    to 6 size v_scale = 2^-129, are multiples of it."""
    n, v_scale = 700, float(np.float32(2.0 ** -138 * 1.359375))
    rng = np.random.RandomState(rows)
    values = np.broadcast_to(4.0 + 2 * (rng.rand(D) < 0.5), (n, D)) * np.sign(rng.randn(D))
    if kind == "e4m3":
        values = values * size
    k, v = stored(kind, sums(rng.randint(0, 8, n) * 0.5), 0x38), stored(kind, values, {1: 0x38, 64: 0x68}[size])
    q = torch.zeros(1, rows, D)
    q[..., :16] = 1
    q = q.to(torch.bfloat16)
    for splits in (0, 1):
        o, _, table, lens = run(fa, kind, sparse, q, k, v, n, 0.125, v_scale=v_scale, num_splits=splits)
        ro, _, weight = paged.decode_paged_any(q[:, None], k, v, table, lens, scale=0.125, v_scale=v_scale)
        tol = (2.0 ** -10 + 1e-3) * weight[:, 0] + 64 * 2.0 ** -149 + 2.0 ** -134
        assert np.all(np.abs(o - ro[:, 0]) <= tol), np.max(np.abs(o - ro[:, 0]) / tol)
