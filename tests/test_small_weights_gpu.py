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
