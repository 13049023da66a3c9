"""Several tokens with a window, in few splits: the rows' bands together are longer than
the window, and may touch one more key tile than a band of the window's length.

Tolerance of an output element, with A = sum p |v| / sum p of its row (fp64): 2^-8 |O|
for the output's rounding to bf16, 2^-8 A for the weights' (half a step each; in 4
bits to f16 and once more with a group scale: 2^-10 and a term below the 1e-6), 1e-3 A
for the scores (512 products in fp32, off by at most 512 * 2^-24 * 2 of sum |q k|
scale, below 16 here), plus 1e-6.  LSE: 1e-3.
"""
import numpy as np
import pytest
import torch

from head_dim_flashattention_gb300 import workloads
from oracle import paged

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def fa(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    import head_dim_flashattention_gb300 as fa
    fa.load_library()
    return fa


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("splits", [0, 1, 2, 3])
@pytest.mark.parametrize("q_len,hq,hk,window", [(16, 2, 2, 32), (8, 4, 2, 64), (4, 8, 2, 31), (2, 4, 4, 32), (5, 3, 1, 1)])
def test_bands_of_several_tokens(fa, q_len, hq, hk, window, splits, kind):
    # every alignment of the band's first position to a tile of 32
    check(fa, [200 + i for i in range(32)] + [q_len, 3], q_len, hq, hk, window, splits, kind)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("q_len,hq,hk", [(3, 8, 4), (16, 1, 1), (1, 8, 4)])
@pytest.mark.parametrize("window", [71, 72, 2 ** 31 - 1])
def test_windows_that_leave_nothing_out(fa, q_len, hq, hk, window, kind):
    check(fa, [2, 1, 0, 13, 71], q_len, hq, hk, window, 0, kind)


def check(fa, lens, q_len, hq, hk, window, splits, kind):
    need = [paged.pages_of(n, PAGE) for n in lens]
    table, at = torch.zeros(len(lens), max(need), dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn(at, PAGE, hk, 512, generator=g) for _ in range(2))
    if kind == "bf16":
        k, v, scales = k.to(torch.bfloat16), v.to(torch.bfloat16), {}
    elif kind == "e2m1":
        k, v = (torch.from_numpy(paged.fp4_rows(x.to(torch.bfloat16), 1.0)) for x in (k, v))
        scales = {"k_scale": 1.0, "v_scale": 1.0}
    else:
        k, v = ((x / 0.04).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        scales = {"k_scale": 0.0371, "v_scale": 0.0517}
    lens = torch.tensor(lens, dtype=torch.int32)
    q = workloads.draft_queries(len(lens), q_len, hq, seed=8)
    f = {"bf16": fa.fa512_decode_paged_q, "e4m3": fa.fa512_decode_paged_fp8, "e2m1": fa.fa512_decode_paged_fp4}[kind]
    out, lse = f(*[x.cuda() for x in (q, k, v, table, lens)], max_kv_len=int(lens.max()), window=window, num_splits=splits,
                 **scales)
    torch.cuda.synchronize()
    assert fa.fa512_device_status() == 0
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    ro, rl, weight = paged.decode_paged_any(q, k, v, table, lens, window=window, **scales)
    assert np.all(np.isfinite(o)) and np.all(np.abs(o - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 1e-3) * weight + 1e-6)
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(l), none) and np.max(np.abs(l[~none] - rl[~none])) <= 1e-3
