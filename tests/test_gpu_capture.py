"""Calls recorded into graphs in ways that a serving loop would: appends with
their quantisation and key bounds, several kinds of call on one schedule, and
schedules of two pools in one graph."""
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


@pytest.mark.parametrize("kv_dtype", ["fp16", "fp8", "fp4"])
def test_appends_are_captured(torch_cuda, kv_dtype):
    """The first append of a pool is recorded into a graph: the rows that its
    buffers hold at replay are stored, bounded, read back, selected and attended to."""
    from prefix_shared_decode_gb300 import select_chunks, sparse_decode_attention
    torch = torch_cuda
    c, D = 32, 128
    x = Cache(torch, 70, kv_dtype, c, D, 2, 2, [40 * c + 3, 30 * c + 9], L=2, ks=0.5, vs=2.0)
    ids = [0, 1]
    q = x.queries(2, 4)
    qd = x.dev(q)
    rows = [[torch.empty((2, 1, 2, D), dtype=torch.float16, device="cuda") for _ in range(2)] for _ in ids]
    lists = torch.empty((2, 2, 6), dtype=torch.int32, device="cuda")
    out = torch.empty_like(qd)
    sched = x.pool.schedule(ids, chunk_lists=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in ids:
            x.pool.append(i, [9 * 10**8 + i], *rows[i])
        select_chunks(x.pool, sched, qd, 6, layer=1, out=lists)
        sparse_decode_attention(x.pool, sched, qd, lists, layer=1, out=out)
    new = [[x.draw(1) for _ in range(2)] for _ in ids]
    for i in ids:
        for dst, src in zip(rows[i], new[i]):
            dst.copy_(torch.from_numpy(src))
        x.k[i], x.v[i] = (np.concatenate([a, b], 1) for a, b in zip((x.k[i], x.v[i]), new[i]))
    for _ in range(2):                          # (the same rows twice are the same rows)
        graph.replay()
        x.check_bounds()
        want = x.want_lists(ids, 1, q, 6, 1, 1)
        np.testing.assert_array_equal(lists.cpu().numpy(), want)
        x.check_attention(out.cpu().numpy(), ids, 1, q, want)
    x.append(0, 1)                              # and eager ones after it
    sched = x.pool.schedule(ids, chunk_lists=True)
    got = select_chunks(x.pool, sched, qd, 6, layer=1)
    x.check_bounds()
    np.testing.assert_array_equal(got.cpu().numpy(), x.want_lists(ids, 1, q, 6, 1, 1))
    assert sched.device_status() == 0


def test_several_calls_on_one_schedule_and_two_pools_in_one_graph(torch_cuda):
    """Whole attention, selection and listed chunks in turn on one schedule,
    layer after layer, between them the same on another pool's: replayed over
    new queries, then eager again, with equal results."""
    from prefix_shared_decode_gb300 import decode_attention, select_chunks, sparse_decode_attention
    torch = torch_cuda
    xs = [Cache(torch, 71, "fp4", 64, 128, 4, 2, [3000, 1500, 700], L=2, shared=300),
          Cache(torch, 72, "fp16", 16, 64, 1, 3, [500, 1, 1300], L=2)]
    ids = [2, 0, 1]
    scheds = [x.pool.schedule(ids, chunk_lists=True) for x in xs]
    qs = [x.dev(x.queries(3, h)) for x, h in zip(xs, (8, 3))]
    bufs = [[[torch.empty_like(q), torch.empty((3, x.Hkv, 5), dtype=torch.int32, device="cuda"), torch.empty_like(q)]
             for _ in range(2)] for x, q in zip(xs, qs)]

    def step():
        for layer in range(2):
            for x, s, q, b in zip(xs, scheds, qs, bufs):
                full, lists, out = b[layer]
                decode_attention(x.pool, s, q, layer=layer, out=full)
                select_chunks(x.pool, s, q, 5, layer=layer, out=lists)
                sparse_decode_attention(x.pool, s, q, lists, layer=layer, out=out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        new = [x.queries(3, h) for x, h in zip(xs, (8, 3))]
        for q, n in zip(qs, new):
            q.copy_(torch.from_numpy(n))
        graph.replay()
        for x, n, b in zip(xs, new, bufs):
            every = np.tile(np.arange(200), (3, x.Hkv, 1))
            for layer in range(2):
                full, lists, out = (t.cpu().numpy() for t in b[layer])
                x.check_attention(full, ids, layer, n, every)
                want = x.want_lists(ids, layer, n, 5, 1, 1)
                np.testing.assert_array_equal(lists, want)
                x.check_attention(out, ids, layer, n, want)
        first = [t.clone() for b in bufs for layer in b for t in layer]
        step()
        assert all(torch.equal(a, t) for a, t in zip(first, (t for b in bufs for layer in b for t in layer)))
    assert all(s.device_status() == 0 for s in scheds)
