"""Waits that run out in the listed chunks' kernel: the call ends, reports it,
and the next call is right."""
import time

import numpy as np
import pytest

from tests.test_gpu_sparse import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.mark.parametrize("kv_dtype,c,D,G", [("fp16", 64, 128, 1), ("fp16", 32, 128, 16), ("fp8", 16, 128, 2),
                                            ("fp4", 16, 64, 4), ("fp4", 32, 128, 12), ("fp4", 64, 128, 8)])
@pytest.mark.parametrize("top_k", [2, 21])
def test_waits_that_run_out(torch_cuda, lib, kv_dtype, c, D, G, top_k):
    """One, two and four groups of warps on the ring; CTAs with one piece and
    with several.  In a stalled call some groups stand at a piece's barriers
    while the waits of others run out, and in other CTAs a single warp has given
    up: all of them meet there and leave together.

    A call ends within 8 limits of about 1 s: the producer's turn, its wait for
    copies in flight (a third of the ring, at most 4 slots) and one for each
    group of the consumers overlap only in part."""
    from prefix_shared_decode_gb300 import sparse_decode_attention
    torch = torch_cuda
    x = Cache(torch, 60 + c + G, kv_dtype, c, D, G, 2, [40 * c + 3, 7, 25 * c, 30 * c + 1])
    ids = [2, 0, 3, 1]
    q = x.queries(len(ids), 2 * G)
    qd = x.dev(q)
    sched = x.pool.schedule(ids, chunk_lists=True)
    lists = np.full((len(ids), 2, top_k), -1, np.int32)
    for r, i in enumerate(ids):
        n = -(-x.k[i].shape[1] // c)
        for h in range(2):
            some = x.rng.permutation(n)[:top_k]
            lists[r, h, :len(some)] = some
    ld = x.dev(lists)
    first = sparse_decode_attention(x.pool, sched, qd, ld)
    x.check_attention(first.cpu().numpy(), ids, 0, q, lists)
    assert sched.device_status() == 0
    assert lib.ca_sched_inject_stall(sched.handle, 1) == 0
    t0 = time.monotonic()
    sparse_decode_attention(x.pool, sched, qd, ld)
    assert sched.device_status() == -8
    assert time.monotonic() - t0 < 10
    # the units' counters are where they were: the next call merges the same
    # pieces to the same bits
    for _ in range(3):
        assert torch.equal(sparse_decode_attention(x.pool, sched, qd, ld), first)
    assert sched.device_status() == 0


def test_a_stalled_call_leaves_the_counters_at_zero(torch_cuda, lib):
    """Without the status having been read (which clears them too)."""
    from prefix_shared_decode_gb300 import sparse_decode_attention
    torch = torch_cuda
    x = Cache(torch, 61, "fp4", 16, 128, 2, 2, [3000, 800])
    q = x.queries(2, 4)
    qd = x.dev(q)
    sched = x.pool.schedule([0, 1], chunk_lists=True)
    ld = torch.arange(48, dtype=torch.int32, device="cuda").expand(2, 2, 48).contiguous()
    first = sparse_decode_attention(x.pool, sched, qd, ld)
    assert lib.ca_sched_inject_stall(sched.handle, 1) == 0
    sparse_decode_attention(x.pool, sched, qd, ld)
    assert torch.equal(sparse_decode_attention(x.pool, sched, qd, ld), first)
    assert sched.device_status() == -8
    assert torch.equal(sparse_decode_attention(x.pool, sched, qd, ld), first)


def test_more_pieces_than_one_to_a_cta(torch_cuda, lib):
    """A CTA that gives up in its first piece goes on through all of them."""
    from prefix_shared_decode_gb300 import sparse_decode_attention
    torch = torch_cuda
    b, H = 64, 32
    x = Cache(torch, 62, "fp16", 32, 64, 1, H, [3 + i for i in range(b)])
    q = x.queries(b, H)
    qd = x.dev(q)
    sched = x.pool.schedule(list(range(b)), chunk_lists=True)
    ld = torch.zeros((b, H, 1), dtype=torch.int32, device="cuda")
    first = sparse_decode_attention(x.pool, sched, qd, ld)
    x.check_attention(first.cpu().numpy(), list(range(b)), 0, q, np.zeros((b, H, 1), np.int64))
    assert lib.ca_sched_inject_stall(sched.handle, 1) == 0
    sparse_decode_attention(x.pool, sched, qd, ld)
    assert sched.device_status() == -8
    assert torch.equal(sparse_decode_attention(x.pool, sched, qd, ld), first)
    assert sched.device_status() == 0
