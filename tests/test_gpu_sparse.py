"""Chunk selection and attention over listed chunks on the GPU, for every pool
type: key bounds bit for bit, selected chunks equal to the 64-bit ranking
(ties and scores that 32 bits cannot tell apart among them), outputs against
the fp64 definition over the listed chunks' stored values.

Tolerance of an output: as for the 4-bit pool's attention (tests/
test_gpu_fp4.py): half a step of fp16, the fp16 weights' 2^-11 * A with
A = sum p|v|, and 2^-12 * A for everything held in 32 bits."""
import numpy as np
import pytest

from oracle import fp4 as F4
from oracle import fp8 as F8
from oracle import sparse as SP
from tests.test_gpu_fp4 import near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def held(x, kv_dtype, S):
    """Stored values of fp16 rows, float64."""
    if kv_dtype == "fp16":
        return x.astype(np.float64)
    return F8.dequantize(F8.quantize(x, S), S) if kv_dtype == "fp8" else F4.roundtrip(x, S)


class Cache:
    def __init__(self, torch, seed, kv_dtype, c, D, G, Hkv, lens, L=1, ks=1.0, vs=1.0, shared=0, rows=None):
        from prefix_shared_decode_gb300 import Pool
        self.torch, self.rng = torch, np.random.default_rng(seed)
        self.kv_dtype, self.c, self.D, self.L, self.Hkv, self.ks, self.vs = kv_dtype, c, D, L, Hkv, ks, vs
        self.pool = Pool(L, Hkv * G, D, c, sum(-(-n // c) for n in lens) + 40, n_kv_heads=Hkv, kv_dtype=kv_dtype,
                         k_scale=ks, v_scale=vs, chunk_bounds=True)
        self.k, self.v = [], []
        first = None
        for i, n in enumerate(lens):
            k, v = (self.draw(n) for _ in range(2)) if rows is None else rows[i]
            m = min(shared, n)
            if first is not None and m:
                k[:, :m], v[:, :m] = first[0][:, :m], first[1][:, :m]
            first = first or (k, v)
            self.k.append(k)
            self.v.append(v)
            self.pool.insert(i, list(range(m)) + [10**6 * (i + 1) + j for j in range(n - m)], self.dev(k), self.dev(v))

    def draw(self, n):
        x = self.rng.standard_normal((self.L, n, self.Hkv, self.D)) + self.rng.standard_normal((1, 1, self.Hkv, self.D))
        return x.astype(np.float16)

    def dev(self, x):
        return self.torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def append(self, i, n):
        k, v = self.draw(n), self.draw(n)
        self.k[i], self.v[i] = np.concatenate([self.k[i], k], 1), np.concatenate([self.v[i], v], 1)
        self.pool.append(i, [5 * 10**8 + i * 1000 + self.k[i].shape[1] + j for j in range(n)], self.dev(k), self.dev(v))

    def bounds(self, i, layer):
        return SP.bounds(held(self.k[i][layer], self.kv_dtype, self.ks), self.c)

    def check_bounds(self):
        got = self.pool.bounds_view().cpu().numpy()
        for i in range(len(self.k)):
            slots = self.pool.seq_slots(i)
            for layer in range(self.L):
                unit = float(np.float32(self.ks)) if self.kv_dtype != "fp16" else 1.0
                np.testing.assert_array_equal(got[slots, layer].astype(np.float64), self.bounds(i, layer) / unit)

    def queries(self, b, H):
        return self.rng.standard_normal((b, H, self.D)).astype(np.float16)

    def want_lists(self, ids, layer, q, top_k, sink, recent):
        return np.stack([[SP.select(s, top_k, sink, recent) for s in SP.scores(q[r], self.bounds(i, layer))]
                         for r, i in enumerate(ids)])

    def check_attention(self, got, ids, layer, q, lists, scale=None):
        scale = scale or 1 / np.sqrt(self.D)
        for r, i in enumerate(ids):
            k = held(self.k[i][layer], self.kv_dtype, self.ks)
            v = held(self.v[i][layer], self.kv_dtype, self.vs)
            want = SP.attention(q[r], k, v, lists[r], self.c, scale)
            near(got[r], want, SP.attention(q[r], k, np.abs(v), lists[r], self.c, scale))


POOLS = [("fp16", 16, 64, 1, 2), ("fp16", 64, 128, 4, 2), ("fp16", 32, 256, 2, 1), ("fp16", 16, 256, 12, 1),
         ("fp16", 64, 128, 16, 1), ("fp16", 32, 128, 64, 1), ("fp8", 64, 128, 1, 3), ("fp8", 16, 128, 8, 1),
         ("fp8", 32, 128, 9, 1), ("fp4", 64, 128, 1, 3), ("fp4", 16, 64, 4, 2), ("fp4", 32, 128, 16, 1),
         ("fp4", 64, 64, 3, 2), ("fp16", 32, 64, 8, 2), ("fp4", 16, 64, 1, 2),
         ("fp4", 32, 128, 1, 1)]


@pytest.mark.parametrize("kv_dtype,c,D,G,Hkv", POOLS)
def test_a_step_over_selected_chunks(torch_cuda, kv_dtype, c, D, G, Hkv):
    """Select and attend as a decode step does, over contexts from one token
    on, with a shared prefix, before and after appends."""
    from prefix_shared_decode_gb300 import decode_attention, select_chunks, sparse_decode_attention
    torch = torch_cuda
    lens = [1, c, 5 * c + 3, 17 * c, 40 * c + 7, 3 * c - 1, 33 * c + 1]
    x = Cache(torch, c + D + G, kv_dtype, c, D, G, Hkv, lens, L=2, ks=0.75, vs=1.25, shared=2 * c + 5)
    ids = [4, 0, 2, 6, 1, 5, 3]
    q = x.queries(len(ids), Hkv * G)
    qd = x.dev(q)
    for step in range(3):
        x.check_bounds()
        sched = x.pool.schedule(ids, chunk_lists=True)
        for layer, top_k, sink, recent in ((1, 7, 1, 1), (0, 1, 0, 1), (1, 4, 0, 0), (0, 12, 3, 4), (1, 41, 1, 2)):
            got = select_chunks(x.pool, sched, qd, top_k, layer=layer, sink=sink, recent=recent)
            want = x.want_lists(ids, layer, q, top_k, sink, recent)
            np.testing.assert_array_equal(got.cpu().numpy(), want)
            out = sparse_decode_attention(x.pool, sched, qd, got, layer=layer).cpu().numpy()
            x.check_attention(out, ids, layer, q, want)
        # every chunk listed: ordinary decode attention
        every = select_chunks(x.pool, sched, qd, 60)
        full = decode_attention(x.pool, sched, qd).cpu().numpy()
        x.check_attention(full, ids, 0, q, every.cpu().numpy())
        x.check_attention(sparse_decode_attention(x.pool, sched, qd, every).cpu().numpy(), ids, 0, q, every.cpu().numpy())
        assert sched.device_status() == 0
        for i in ids:
            x.append(i, (1, c + 2)[step % 2])


@pytest.mark.parametrize("kv_dtype,D,b,n", [("fp16", 64, 1, 40000), ("fp8", 128, 2, 20000), ("fp4", 64, 1, 100000),
                                            ("fp16", 128, 40, 900)])
def test_long_contexts_and_wide_batches(torch_cuda, kv_dtype, D, b, n):
    """Contexts whose chunks several CTAs score and read, and batches whose
    pairs fill the card with one CTA each."""
    from prefix_shared_decode_gb300 import select_chunks, sparse_decode_attention
    x = Cache(torch_cuda, n + b, kv_dtype, 16, D, 2, 1 if b == 1 else 4, [n - 3 * i for i in range(b)])
    ids = list(range(b))
    q = x.queries(b, x.Hkv * 2)
    qd = x.dev(q)
    sched = x.pool.schedule(ids, chunk_lists=True)
    for top_k in (1, 33, 500):
        got = select_chunks(x.pool, sched, qd, top_k)if top_k > 1 else select_chunks(x.pool, sched, qd, 1, sink=0)
        want = x.want_lists(ids, 0, q, top_k, 0 if top_k == 1 else 1, 1)
        np.testing.assert_array_equal(got.cpu().numpy(), want)
        x.check_attention(sparse_decode_attention(x.pool, sched, qd, got).cpu().numpy(), ids, 0, q, want)
    assert sched.device_status() == 0


@pytest.mark.parametrize("n_chunks", [40, 700, 3000])
def test_ties_go_to_the_lower_chunk(torch_cuda, n_chunks):
    """Equal chunks, queries of zeros, and chunks that differ by less than a
    32-bit sum can hold: among few and among more than 256 near-equal ones."""
    from prefix_shared_decode_gb300 import select_chunks
    torch = torch_cuda
    rng = np.random.default_rng(n_chunks)
    c, D = 16, 64
    base = rng.standard_normal((1, c, 1, D)).astype(np.float16)
    k = np.tile(base, (1, n_chunks, 1, 1))
    big = rng.permutation(n_chunks)[:5]
    for j in big:                                  # a few larger ones among the equal
        k[0, j * c, 0, 3] += 2 + 0.25 * (j % 7)
    x = Cache(torch, 1, "fp16", c, D, 2, 1, [n_chunks * c], rows=[(k, k)])
    q = x.queries(1, 2)
    q[:, :, 3] = 1
    near_ = k.copy()
    # chunk j's score grows by j % 5 steps of 2^-24 * 2^-8: fp32 sums near 50 end at 2^-19
    near_[0, ::c, 0, 0] = 1024
    near_[0, ::c, 0, 1] = ((np.arange(n_chunks) * 3) % 5 + 1) * 2.0 ** -24
    near_[0, 1::c, 0, 1] = -1
    y = Cache(torch, 2, "fp16", c, D, 2, 1, [n_chunks * c], rows=[(near_, near_)])
    qn = np.zeros((1, 2, D), np.float16)
    qn[0, 0, 0], qn[0, 0, 1] = 8, 2.0 ** -8
    qn[0, 1, 0] = -1
    for cache, qq in ((x, q), (x, np.zeros_like(q)), (y, qn), (y, -q)):
        sched = cache.pool.schedule([0], chunk_lists=True)
        for top_k, sink, recent in ((1, 0, 0), (9, 1, 1), (n_chunks // 2, 0, 3), (n_chunks - 1, 2, 2)):
            got = select_chunks(cache.pool, sched, cache.dev(qq), top_k, sink=sink, recent=recent).cpu().numpy()
            np.testing.assert_array_equal(got, cache.want_lists([0], 0, qq, top_k, sink, recent))


def test_queries_that_are_not_finite(torch_cuda):
    """No score to go by: still top_k distinct chunks, the forced among them."""
    from prefix_shared_decode_gb300 import select_chunks
    torch = torch_cuda
    x = Cache(torch, 3, "fp16", 16, 64, 2, 1, [16 * 300])
    sched = x.pool.schedule([0], chunk_lists=True)
    for bad in (np.inf, -np.inf, np.nan):
        q = x.queries(1, 2)
        q[0, 1, 5] = bad
        got = select_chunks(x.pool, sched, x.dev(q), 20, sink=2, recent=2).cpu().numpy()[0, 0]
        assert (np.diff(got) > 0).all() and got[0] == 0 and got[1] == 1 and got[-1] == 299 and got[-2] == 298
    assert sched.device_status() == 0


def test_lists_of_any_order(torch_cuda):
    """Unordered lists, skipped entries, a chunk twice, an empty list (zeros),
    an entry past the context (skipped and reported)."""
    from prefix_shared_decode_gb300 import sparse_decode_attention
    torch = torch_cuda
    x = Cache(torch, 4, "fp4", 32, 128, 4, 2, [700, 33, 1000])
    ids = [0, 1, 2]
    q = x.queries(3, 8)
    qd = x.dev(q)
    sched = x.pool.schedule(ids, chunk_lists=True)
    lists = np.full((3, 2, 9), -1, np.int32)
    lists[0, 0, :6] = [7, 3, 21, 0, 5, 4]
    lists[0, 1, 3:] = [5, 5, 9, 5, 21, -7]
    lists[1, 0, ::4] = [1, 0, -1]
    lists[2, 1] = [31, 30, 29, 3, 2, 1, 0, 11, 10]
    out = torch.full((4, 8, 128), 7.0, dtype=torch.float16, device="cuda")
    got = sparse_decode_attention(x.pool, sched, qd, torch.from_numpy(lists).cuda(), out=out[:3]).cpu().numpy()
    x.check_attention(got, ids, 0, q, lists)
    assert (got[1, 4:] == 0).all() and (got[2, :4] == 0).all()
    assert (out[3] == 7).all()
    assert sched.device_status() == 0
    lists[1, 0, 0] = 2                                      # sequence 1 has chunks 0 and 1
    got = sparse_decode_attention(x.pool, sched, qd, torch.from_numpy(lists).cuda()).cpu().numpy()
    assert sched.device_status() == -7
    lists[1, 0, 0] = -1
    x.check_attention(got, ids, 0, q, lists)
    assert sched.device_status() == 0
    # a scale of the caller's own
    got = sparse_decode_attention(x.pool, sched, qd, torch.from_numpy(lists).cuda(), scale=0.3).cpu().numpy()
    x.check_attention(got, ids, 0, q, lists, 0.3)


def test_graph_and_streams(torch_cuda):
    """Both calls captured and replayed over appends in place; the same calls
    issued on two other streams at once, each on a schedule of its own."""
    from prefix_shared_decode_gb300 import select_chunks, sparse_decode_attention
    torch = torch_cuda
    x = Cache(torch, 5, "fp8", 64, 128, 4, 2, [3000, 5003, 64 * 30 + 1])
    ids = [0, 1, 2]
    q = x.queries(3, 8)
    qd = x.dev(q)
    sched = x.pool.schedule(ids, chunk_lists=True)
    lists = torch.empty((3, 2, 6), dtype=torch.int32, device="cuda")
    out = torch.empty_like(qd)

    def step():
        select_chunks(x.pool, sched, qd, 6, out=lists)
        sparse_decode_attention(x.pool, sched, qd, lists, out=out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for i in ids:
            x.append(i, 1)
        q = x.queries(3, 8)
        qd.copy_(torch.from_numpy(q))
        lists.fill_(-5)
        graph.replay()
        want = x.want_lists(ids, 0, q, 6, 1, 1)
        np.testing.assert_array_equal(lists.cpu().numpy(), want)
        x.check_attention(out.cpu().numpy(), ids, 0, q, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    scheds = [x.pool.schedule(ids, chunk_lists=True) for _ in streams]
    got = []
    torch.cuda.synchronize()
    for _ in range(10):
        for s, sc in zip(streams, scheds):
            a = select_chunks(x.pool, sc, qd, 6, stream=s)
            got.append((a, sparse_decode_attention(x.pool, sc, qd, a, stream=s)))
    torch.cuda.synchronize()
    for a, o in got:
        assert torch.equal(a, lists) and torch.equal(o, out)
    assert all(s.device_status() == 0 for s in [sched, *scheds])


@pytest.mark.parametrize("kv_dtype,G,D", [("fp16", 4, 128), ("fp4", 64, 64), ("fp16", 32, 256)])
def test_channels_of_large_keys(torch_cuda, kv_dtype, G, D):
    """A few channels a hundred times the others', as models' keys have: the
    order among the chunks is still that of the exact scores."""
    from prefix_shared_decode_gb300 import select_chunks
    c = 16
    x = Cache(torch_cuda, 40 + G, kv_dtype, c, D, G, 1, [1], rows=[(np.zeros((1, 1, 1, D), np.float16),) * 2])
    k = x.draw(900 * c)
    k[..., 3] += 300
    k[..., D // 2] *= 60
    x = Cache(torch_cuda, 41 + G, kv_dtype, c, D, G, 1, [900 * c], rows=[(k, k)])
    q = x.queries(1, G)
    sched = x.pool.schedule([0], chunk_lists=True)
    for top_k in (5, 64, 400):
        got = select_chunks(x.pool, sched, x.dev(q), top_k).cpu().numpy()
        np.testing.assert_array_equal(got, x.want_lists([0], 0, q, top_k, 1, 1))


def test_the_longest_contexts(torch_cuda):
    """49152 chunks are scored; one more is refused, while lists of the
    caller's own still reach every chunk."""
    from prefix_shared_decode_gb300 import CAError, Pool, select_chunks, sparse_decode_attention
    torch = torch_cuda
    c, D, n = 16, 64, 49152 * 16
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn((1, n + 1, 1, D), generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    pool = Pool(1, 1, D, c, 49160, chunk_bounds=True)
    pool.insert(0, np.arange(n), k[:, :n].contiguous(), v[:, :n].contiguous())
    q = torch.randn((1, 1, D), generator=g, device="cuda", dtype=torch.float16)
    sched = pool.schedule([0], chunk_lists=True)
    got = select_chunks(pool, sched, q, 100, sink=2, recent=3).cpu().numpy()[0, 0]
    bnd = k[0, :n, 0].view(-1, c, D).double()
    qd = q[0, 0].double()
    score = torch.maximum(qd * bnd.amax(1), qd * bnd.amin(1)).sum(-1).cpu().numpy()
    np.testing.assert_array_equal(got, SP.select(score, 100, 2, 3))
    pool.append(0, [n], k[:, n:].contiguous(), v[:, n:].contiguous())
    sched = pool.schedule([0], chunk_lists=True)
    with pytest.raises(CAError) as e:
        select_chunks(pool, sched, q, 100)
    assert e.value.name == "CA_ERR_UNSUPPORTED"
    lists = torch.tensor([[[49152, 7]]], dtype=torch.int32, device="cuda")
    out = sparse_decode_attention(pool, sched, q, lists).cpu().numpy()
    rows = list(range(7 * c, 8 * c)) + [n]
    kk, vv = (t[0, rows].cpu().numpy().astype(np.float64) for t in (k, v))
    want = SP.attention(q[0].cpu().numpy(), kk, vv, [[0, 1]], c, D ** -0.5)
    near(out[0], want, SP.attention(q[0].cpu().numpy(), kk, np.abs(vv), [[0, 1]], c, D ** -0.5))
    assert sched.device_status() == 0


def test_captured_before_any_call(torch_cuda):
    """A graph whose capture is the pool's first use of both calls, and two
    runs of the same lists that agree bit for bit however the pieces arrive."""
    from prefix_shared_decode_gb300 import select_chunks, sparse_decode_attention
    torch = torch_cuda
    x = Cache(torch, 8, "fp4", 32, 64, 2, 1, [2000, 1777])
    q = x.queries(2, 2)
    qd = x.dev(q)
    sched = x.pool.schedule([1, 0], chunk_lists=True)
    lists = torch.empty((2, 1, 40), dtype=torch.int32, device="cuda")
    out = torch.empty_like(qd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        select_chunks(x.pool, sched, qd, 40, out=lists)
        sparse_decode_attention(x.pool, sched, qd, lists, out=out)
    graph.replay()
    want = x.want_lists([1, 0], 0, q, 40, 1, 1)
    np.testing.assert_array_equal(lists.cpu().numpy(), want)
    x.check_attention(out.cpu().numpy(), [1, 0], 0, q, want)
    first = out.clone()
    for _ in range(20):
        graph.replay()
        assert torch.equal(out, first)


def test_flat_pools_and_wide_lists(torch_cuda):
    """A pool without sharing; lists wider than any context; one entry."""
    from prefix_shared_decode_gb300 import Pool, select_chunks, sparse_decode_attention
    torch = torch_cuda
    rng = np.random.default_rng(9)
    c, D, L = 16, 128, 3
    pool = Pool(L, 2, D, c, 60, no_sharing=True, kv_dtype="fp8", chunk_bounds=True)
    k, v = rng.standard_normal((2, L, 200, 2, D)).astype(np.float16)
    dk, dv = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    for i in range(3):
        pool.insert(i, list(range(200)), dk, dv)
    sched = pool.schedule([2, 0, 1], chunk_lists=True)
    q = rng.standard_normal((3, 2, D)).astype(np.float16)
    qd = torch.from_numpy(q).cuda()
    hk, hv = held(k, "fp8", 1.0), held(v, "fp8", 1.0)
    for top_k in (1000, 13, 1):
        lists = select_chunks(pool, sched, qd, top_k, layer=2, sink=0)
        got = sparse_decode_attention(pool, sched, qd, lists, layer=2).cpu().numpy()
        lists = lists.cpu().numpy()
        for r in range(3):
            want = [SP.select(s, top_k, 0, 1) for s in SP.scores(q[r], SP.bounds(hk[2], c))]
            np.testing.assert_array_equal(lists[r], want)
            near(got[r], SP.attention(q[r], hk[2], hv[2], want, c, D ** -0.5),
                 SP.attention(q[r], hk[2], np.abs(hv[2]), want, c, D ** -0.5))
    assert sched.device_status() == 0


def test_refusals(torch_cuda, lib):
    from prefix_shared_decode_gb300 import CAError, Pool, select_chunks, sparse_decode_attention
    torch = torch_cuda
    x = Cache(torch, 6, "fp16", 16, 64, 2, 2, [100, 50])
    sched = x.pool.schedule([0, 1], chunk_lists=True)
    q = x.dev(x.queries(2, 4))
    lists = select_chunks(x.pool, sched, q, 3)
    stream = torch.cuda.current_stream().cuda_stream
    a = (x.pool.handle, sched.handle)
    assert lib.ca_select_chunks(*a, 1, q.data_ptr(), 3, 1, 1, lists.data_ptr(), stream) == -1       # layer
    assert lib.ca_select_chunks(*a, 0, q.data_ptr(), 0, 0, 0, lists.data_ptr(), stream) == -1       # top_k
    assert lib.ca_select_chunks(*a, 0, q.data_ptr(), 3, 2, 2, lists.data_ptr(), stream) == -1       # sink + recent
    assert lib.ca_select_chunks(*a, 0, q.data_ptr(), 3, -1, 1, lists.data_ptr(), stream) == -1
    assert lib.ca_select_chunks(*a, 0, q.data_ptr() + 2, 3, 1, 1, lists.data_ptr(), stream) == -1   # alignment
    assert lib.ca_select_chunks(*a, 0, None, 3, 1, 1, lists.data_ptr(), stream) == -1
    assert lib.ca_sparse_attention(*a, 0, q.data_ptr(), lists.data_ptr(), 3, None, 1.0, stream) == -1
    assert lib.ca_sparse_attention(*a, 0, q.data_ptr(), None, 3, q.data_ptr(), 1.0, stream) == -1
    assert lib.ca_sparse_attention(*a, 0, q.data_ptr(), lists.data_ptr(), 2**31 - 1, q.data_ptr(), 1.0, stream) == -9
    for bad in (lambda: select_chunks(x.pool, x.pool.schedule([0, 1]), q, 3),
                lambda: select_chunks(x.pool, sched, q, 1), lambda: select_chunks(x.pool, sched, q[:1], 3),
                lambda: select_chunks(x.pool, sched, q.float(), 3), lambda: select_chunks(x.pool, sched, q.cpu(), 3),
                lambda: select_chunks(x.pool, sched, q, 3, out=lists[..., :2]),
                lambda: sparse_decode_attention(x.pool, sched, q, lists.long()),
                lambda: sparse_decode_attention(x.pool, sched, q, lists[:1]),
                lambda: sparse_decode_attention(x.pool, sched, q, lists.cpu()),
                lambda: sparse_decode_attention(x.pool, sched, q, lists[..., :0]),
                lambda: sparse_decode_attention(x.pool, sched, q.transpose(0, 1), lists)):
        with pytest.raises(ValueError):
            bad()

    def refused(name, fn):
        with pytest.raises(CAError) as e:
            fn()
        assert e.value.name == name

    multi = x.pool.schedule([0, 1], q_len=2, chunk_lists=True)
    refused("CA_ERR_UNSUPPORTED", lambda: sparse_decode_attention(x.pool, multi, q, lists))
    plain = Pool(1, 4, 64, 16, 20, n_kv_heads=2)
    t = torch.zeros((1, 40, 2, 64), dtype=torch.float16, device="cuda")
    plain.insert(0, list(range(40)), t, t)
    with pytest.raises(ValueError):
        plain.bounds_view()
    ps = plain.schedule([0], chunk_lists=True)
    refused("CA_ERR_INVALID", lambda: select_chunks(plain, ps, q[:1], 3))
    # lists of the caller's own need no bounds
    sparse_decode_attention(plain, ps, q[:1], torch.zeros((1, 2, 1), dtype=torch.int32, device="cuda"))
    x.append(0, 40)
    refused("CA_ERR_STALE", lambda: select_chunks(x.pool, sched, q, 3))
    refused("CA_ERR_STALE", lambda: sparse_decode_attention(x.pool, sched, q, lists))


def test_lists_whose_indexes_would_overflow(torch_cuda, lib):
    """Refused on the host: a single row's list within a step of 2^31 entries."""
    from prefix_shared_decode_gb300 import kernel_launches
    x = Cache(torch_cuda, 7, "fp16", 16, 64, 1, 1, [100])
    sched = x.pool.schedule([0], chunk_lists=True)
    q = x.dev(x.queries(1, 1))
    stream = torch_cuda.cuda.current_stream().cuda_stream
    a = (x.pool.handle, sched.handle, 0, q.data_ptr())
    before = kernel_launches()
    for k in (2**31 - 1, 2**31 - 256):
        assert lib.ca_select_chunks(*a, k, 0, 0, q.data_ptr(), stream) == -9
        assert lib.ca_sparse_attention(*a, q.data_ptr(), k, q.data_ptr(), 1.0, stream) == -9
    assert kernel_launches() == before
