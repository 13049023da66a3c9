"""Calls on another stream than the current one: what a call allocates for
itself must not come from a block that the current stream still uses."""
import pytest
import torch

from head_dim_flashattention_gb300 import _binding, workloads

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
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(*shape, seed=1):
    return workloads.randn_bf16(shape, seed).cuda()


def cache(fp8=False, layers=()):
    k = rows(*layers, 40, 64, 4, D, seed=2)
    return (k.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else k), torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)


def prefill(fa, d):
    q, k = rows(300, 8, d), rows(300, 4, d, seed=2)
    f = fa.fa512_prefill if d == D else fa.fa512_prefill_d256
    return lambda **kw: f(q, k, k, **kw)


def prefill_paged(fa):
    k, pt = cache()
    q, cu, used = rows(200, 8, D), i32([0, 120, 200]), i32([1000, 900])
    return lambda **kw: fa.fa512_prefill_paged(q, k, k, pt, cu, used, max_seqlen_q=120, **kw)


def decode(fa, f, q_len, fp8=False):
    k, pt = cache(fp8)
    q, n = rows(2, *([q_len] if q_len else []), 8, D), i32([1200, 900])
    return lambda **kw: f(q, k, k, pt, n, **kw)


def compact(fa):
    k, pt = cache()
    n, acc, na = i32([1200, 900]), i32([[1, 3], [0, 2]]), i32([2, 1])
    return lambda **kw: (fa.fa512_cache_compact(k, k, pt, n, acc, na, q_len=5, **kw),)


def fork(fa):
    k, pt = cache(layers=(1,))
    n, par, refs = i32([1200, 640]), i32([0, 1, 1]), torch.ones(40, dtype=torch.int32, device="cuda")
    return lambda **kw: fa.fa512_cache_fork(k, k, pt, n, par, refs, **kw)


def resize(fa):
    pt = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    a, z, refs = i32([1200, 900]), i32([700, 901]), torch.ones(40, dtype=torch.int32, device="cuda")
    return lambda **kw: fa.fa512_cache_resize(pt, a, z, refs, page_size=64, **kw)


CALLS = {
    "prefill": lambda fa: prefill(fa, 512), "prefill_d256": lambda fa: prefill(fa, 256),
    "prefill_paged": prefill_paged,
    "decode": lambda fa: decode(fa, fa.fa512_decode_paged, 0),
    "decode_q": lambda fa: decode(fa, fa.fa512_decode_paged_q, 3),
    "decode_fp8": lambda fa: decode(fa, fa.fa512_decode_paged_fp8, 3, True),
    "tree": lambda fa: decode(fa, fa.fa512_decode_paged_tree, 9),
    "tree_fp8": lambda fa: decode(fa, fa.fa512_decode_paged_tree_fp8, 40, True),
    "compact": compact, "fork": fork, "resize": resize,
}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_outputs_are_not_taken_from_blocks_in_use(fa, name, raw):
    """The current stream has yet to write tensors that were given back to the
    allocator, of the sizes of the outputs; the call on a side stream finishes before it does."""
    run = CALLS[name](fa)
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.empty_like(t) for t in want for _ in range(2)]
    torch.cuda._sleep(40_000_000)
    for t in freed:
        t.fill_(9)
    del freed, t
    got = run(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert fa.fa512_device_status() == 0
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_allocations_belong_to_the_stream_of_the_call(cuda_device):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = torch.empty(3 << 20, dtype=torch.uint8, device="cuda")
    at = a.data_ptr()
    del a
    t = _binding._new(_binding._side(side), 3 << 20, torch.uint8, cuda_device)
    assert t.data_ptr() != at
    u = _binding._new(_binding._side(torch.cuda.current_stream()), 3 << 20, torch.uint8, cuda_device)
    assert u.data_ptr() == at
    # a handle of 0 is the default stream, also while another one is current
    with torch.cuda.stream(side):
        assert _binding._side(0) == torch.cuda.default_stream() and _binding._side(side.cuda_stream) is None


def test_results_of_a_side_stream_outlive_their_readers_here(fa):
    """A returned tensor that is dropped while the current stream still reads it is not handed to the side stream."""
    run = CALLS["tree"](fa)
    want = run()[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(40_000_000)
    copy = out + 0
    del out, lse
    with torch.cuda.stream(side):
        junk = [torch.full_like(want, 9) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(junk) == 4


@pytest.mark.parametrize("name", ["decode", "fork", "resize", "tree"])
def test_a_side_stream_inside_a_capture(fa, name):
    """The call's own tensors belong to the graph: replays find them, and later allocations do not."""
    run = CALLS[name](fa)
    want = [t.clone() for t in run()]
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        junk = [torch.full_like(t, 9) for t in want for _ in range(4)]
        for t in got:
            t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.all(t == 9) for t in junk)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert fa.fa512_device_status() == 0
