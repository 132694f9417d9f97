"""Calls that are given a stream of their own: what they allocate is ordered on
that stream, whatever the current stream still has to do."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

LATE = 200_000_000          # clock cycles: some 0.1 s


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.fixture(scope="module")
def cache(torch_cuda):
    from prefix_shared_decode_gb300 import Pool
    torch = torch_cuda
    g = torch.Generator("cuda").manual_seed(5)
    pool = Pool(2, 8, 128, 64, 200, n_kv_heads=2, chunk_bounds=True)
    k, v = (torch.randn((2, 3000, 2, 128), generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    for i in range(3):
        pool.insert(i, np.arange(3000) + 10**6 * i, k, v)
    q = torch.randn((3, 8, 128), generator=g, device="cuda", dtype=torch.float16)
    lists = torch.arange(12, dtype=torch.int32, device="cuda").expand(3, 2, 12).contiguous()
    torch.cuda.synchronize()
    return pool, q, lists


def calls(pool, q, lists):
    from prefix_shared_decode_gb300 import decode_attention, select_chunks, sparse_decode_attention
    return {
        "decode": lambda sched, s: [decode_attention(pool, sched, q, stream=s)],
        "select": lambda sched, s: [select_chunks(pool, sched, q, 12, stream=s)],
        "sparse": lambda sched, s: [sparse_decode_attention(pool, sched, q, lists, stream=s)],
        "read": lambda sched, s: list(pool.read_batch([1, 0], [64, 0], [900, 2000], stream=s)),
    }


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("name", ["decode", "select", "sparse", "read"])
def test_results_are_the_streams_own(torch_cuda, cache, name, form):
    """Blocks of the results' sizes are freed while the current stream is still
    to write them: a result that lay in one of them would be overwritten."""
    torch = torch_cuda
    pool, q, lists = cache
    fn = calls(pool, q, lists)[name]
    sched = pool.schedule([0, 1, 2], chunk_lists=True)
    want = [t.clone() for t in fn(sched, None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty_like(t) for t in want for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(LATE)
    for t in old:
        t.fill_(77)
    held = {t.data_ptr() for t in old}
    del old, t
    got = fn(sched, side if form == "stream" else side.cuda_stream)
    assert not held & {t.data_ptr() for t in got}
    side.synchronize()
    assert all(torch.equal(a.cpu(), b.cpu()) for a, b in zip(got, want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # dropped at once, with the stream still to write it: the current stream is
    # not given the memory
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
    got = fn(sched, side)
    held = {t.data_ptr() for t in got}
    del got
    new = [torch.full_like(t, 3) for t in want for _ in range(2)]
    assert not held & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    assert all((t == 3).all() for t in new)
    # the default stream by its handle, 0
    got = fn(sched, 0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_workspace_is_filled_on_the_calls_stream(torch_cuda, cache):
    """A schedule's first call, on a side stream: its new workspace is not
    cleared by a fill that the current stream gets to after the kernels; and a
    larger one that replaces it leaves the old memory alone until they are done."""
    from prefix_shared_decode_gb300 import decode_attention
    torch = torch_cuda
    pool, q, _ = cache
    want = decode_attention(pool, pool.schedule([0, 1, 2]), q)
    side = torch.cuda.Stream()
    sched = pool.schedule([0, 1, 2])
    torch.cuda.synchronize()
    torch.cuda._sleep(LATE)
    got = decode_attention(pool, sched, q, stream=side)
    side.synchronize()
    assert torch.equal(got.cpu(), want.cpu())
    torch.cuda.synchronize()
    assert sched._ws.any() and torch.equal(got, want)
    # used by another stream: its memory is not handed on while that one works
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        torch.cuda._sleep(LATE)
    got = decode_attention(pool, sched, q, stream=other)
    at, n = sched._ws.data_ptr(), sched._ws.numel()
    sched._ws = None
    with torch.cuda.stream(side):
        new = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert at not in {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    assert torch.equal(got, want)
