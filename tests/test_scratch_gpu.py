"""Calls that make their workspace for themselves, also where PyTorch has no allocation without a tensor."""
import pytest
import torch

from head_dim_flashattention_gb300 import _binding, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa(cuda_device):
    import __graft_entry__
    __graft_entry__.build()
    import head_dim_flashattention_gb300 as fa
    fa.load_library()
    return fa


def calls(fa, **kw):
    """A selection, a decode over lists of it in bf16 and one over a 4-bit cache; several segments a sequence."""
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn(70, 16, 4, 512, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    k4, v4 = (torch.randint(0, 64, (70, 16, 4, 288), generator=gen).to(torch.uint8).cuda() for _ in range(2))
    table = torch.randperm(70, generator=gen).to(torch.int32).view(2, 35).cuda()
    lens = torch.tensor([560, 301], dtype=torch.int32).cuda()
    q = workloads.draft_queries(2, 1, 8, seed=2).cuda()
    bounds = torch.zeros(70, 4, 2, 512, dtype=torch.bfloat16).cuda()
    fa.fa512_cache_page_bounds(k, table, lens, bounds, q_len=560, q_lens=lens)
    torch.cuda.synchronize()
    sel = fa.fa512_select_pages(q, bounds, table, lens, page_size=16, n_select=9, **kw)
    got = (sel,) + fa.fa512_decode_paged_sparse(q, k, v, table, lens, sel, **kw)
    got += fa.fa512_decode_paged_fp4(q, k4, v4, table, lens, **kw)
    torch.cuda.synchronize()
    assert fa.fa512_device_status() == 0
    return got


@pytest.mark.parametrize("missing", [("_raw_alloc", "_raw_free"), ("_raw_alloc",), ("_raw_free",)])
@pytest.mark.parametrize("side", [False, True])
def test_without_raw_allocations(fa, monkeypatch, missing, side):
    want = calls(fa)
    for name in missing:
        monkeypatch.setattr(_binding, name, None)
    kw = {"stream": torch.cuda.Stream()} if side else {}
    for a, b in zip(calls(fa, **kw), want):
        assert torch.equal(a, b)


def test_a_refused_call_gives_its_workspace_back(fa):
    """In as many bytes as it was taken: nothing is left of a thousand refused calls."""
    q = workloads.draft_queries(1, 1, 8, seed=2).cuda()
    k = torch.zeros(4, 16, 4, 288, dtype=torch.uint8).cuda()
    table, lens = torch.zeros(1, 4, dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(1000):
        with pytest.raises(fa.Fa512Error):
            fa.fa512_decode_paged_fp4(q, k, k, table, lens, max_kv_len=65)     # more than the table holds
    assert torch.cuda.memory_allocated() - before < 1 << 20
