"""CPU pins of the rounding bounds that the E4M3 tree kernels state: a bf16 query as two E4M3 terms, a weight as three
E5M2 terms."""
import numpy as np
import torch

import oracle
from oracle import paged


def test_two_e4m3_terms_of_a_query():
    """Scaled so that the row's largest element is in [128, 256): exact from 2^-9 of the largest upward, off by at most
    2^-17 of it below, and that is reached (largest 128, element 2^-3 (1 + 2^-7))."""
    x = torch.arange(1, 0x4380, dtype=torch.int16).view(torch.bfloat16).double().numpy()      # all in (0, 256)
    assert x.max() < 256
    values = oracle.e4m3_table()
    first = values[paged.e4m3_round(x)]
    err = np.abs(x - first - values[paged.e4m3_round(x - first)])
    assert np.all(err[x >= 128 * 2.0 ** -9] == 0) and np.max(err) == 128 * 2.0 ** -17
    assert err[x == 0.125 * (1 + 2.0 ** -7)] == 2.0 ** -10


def test_three_e5m2_terms_of_a_weight():
    """2^11 p for weights p in (0, 2^4]: off by at most 2^-9 of p or 2^-28."""
    g = torch.Generator().manual_seed(5)
    p = torch.exp2(torch.rand(200000, generator=g, dtype=torch.float64) * 44 - 40).float()
    left = p * 2048
    for _ in range(3):
        left = left - left.to(torch.float8_e5m2).float()
    err = left.double().abs() / 2048
    assert torch.all(err <= torch.maximum(p.double() * 2.0 ** -9, torch.full_like(err, 2.0 ** -28)))
