"""Eviction on the GPU, for every pool type: the kept positions, their rows bit
for bit as the pool held them, the weights, and what later calls make of it."""
import numpy as np
import pytest

from oracle import sparse as SP
from oracle import weights as OW
from tests.test_gpu_fp4 import near
from tests.test_gpu_sparse import POOLS, Cache, held

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def sums(x, b, room):
    """Running sums with ties, zeros of both signs, infinities and NaN."""
    w = x.rng.random((x.L, b, x.Hkv, room)).astype(np.float32) ** 8
    w[x.rng.random(w.shape) < 0.3] = 0.0
    w[x.rng.random(w.shape) < 0.1] = -0.0
    w[x.rng.random(w.shape) < 0.1] = 0.25
    w[x.rng.random(w.shape) < 0.02] = np.nan
    w[x.rng.random(w.shape) < 0.01] = np.inf
    w[x.rng.random(w.shape) < 0.01] = -np.inf
    w[x.rng.random(w.shape) < 0.02] = 1e-42
    return w


def rows(x, i):
    """(k, v) uint16 [L, n, Hkv, D] of what the pool gives back of a sequence."""
    return [t.cpu().numpy().view(np.uint16) for t in x.pool.read(i)]


def check(x, ids, new, was, w, budget, sink, recent, kept, out):
    kept, out = kept.cpu().numpy(), out.cpu().numpy()
    for r, (i, j) in enumerate(zip(ids, new)):
        n = was[i][0].shape[1]
        k, v = rows(x, j)
        m = min(n, budget)
        assert k.shape[1] == m
        for layer in range(x.L):
            for h in range(x.Hkv):
                at = OW.kept(w[layer, r, h, :n], budget, sink, recent)
                np.testing.assert_array_equal(kept[layer, r, h], np.concatenate([at, np.full(budget - m, -1)]))
                got = out[layer, r, h]
                np.testing.assert_array_equal(got[:m].view(np.uint32), w[layer, r, h, at].view(np.uint32))
                assert not got[m:].view(np.uint32).any()
                np.testing.assert_array_equal(k[layer, :, h], was[i][0][layer, at, h])
                np.testing.assert_array_equal(v[layer, :, h], was[i][1][layer, at, h])


@pytest.mark.parametrize("kv_dtype,c,D,G,Hkv", POOLS)
def test_in_place_and_apart(torch_cuda, kv_dtype, c, D, G, Hkv):
    torch = torch_cuda
    lens = [40 * c + 7, 1, c, 5 * c + 3, 17 * c, 3 * c - 1, 33 * c + 1]
    x = Cache(torch, c + D + G, kv_dtype, c, D, G, Hkv, lens, L=2, ks=0.75, vs=1.25, shared=2 * c + 5)
    ids = [4, 0, 2, 6, 1, 5, 3]
    room = 41 * c
    was = {i: rows(x, i) for i in ids}
    # apart: 3 c + 5 tokens, a sink of one whole chunk and a half, into new sequences
    w = sums(x, len(ids), room)
    new = [100 + i for i in ids]
    budget, sink, recent = 3 * c + 5, c + c // 2, 3
    wd = x.dev(w)
    free = x.pool.stats()["free_slots"]
    kept, out = x.pool.evict(x.pool.schedule(ids, chunk_lists=True), wd, budget, sink=sink, recent=recent, into=new[:])
    np.testing.assert_array_equal(wd.cpu().numpy().view(np.uint32), w.view(np.uint32))
    check(x, ids, new, was, w, budget, sink, recent, kept, out)
    for i in ids:
        for a, b in zip(rows(x, i), was[i]):
            np.testing.assert_array_equal(a, b)
    x.pool.remove_batch(new)
    assert x.pool.stats()["free_slots"] == free
    # in place, weights too: one sequence at a time where slots are few
    budget, sink, recent = 2 * c + 1, 1, c
    sched = None
    for r, i in enumerate(ids):
        sched = x.pool.schedule([i], chunk_lists=True, reuse=sched)
        mine = wd[:, r:r + 1].contiguous()
        kept, out = x.pool.evict(sched, mine, budget, sink=sink, recent=recent, out=mine)
        assert out is mine
        check(x, [i], [i], was, w[:, r:r + 1], budget, sink, recent, kept, out)
        assert sched.device_status() == 0


@pytest.mark.parametrize("n,budget,sink,recent", [(20_000, 1, 0, 0), (20_000, 19_999, 0, 0), (20_000, 5000, 0, 0), (20_000, 64, 64, 0),
                                                  (20_000, 64, 0, 64), (20_000, 100, 37, 63), (20_000, 8192, 4, 256),
                                                  (2048, 2047, 1, 1), (2049, 1024, 0, 1)])
@pytest.mark.parametrize("kind", ["mixed", "equal", "one_bit", "nan"])
def test_long_rows(torch_cuda, n, budget, sink, recent, kind):
    """Every pass of the choice: rows of many rounds, all of one value, values that
    differ in their last bit, nothing but NaN."""
    from prefix_shared_decode_gb300 import Pool
    x = Cache(torch_cuda, 3, "fp16", 64, 64, 1, 2, [n])
    x.pool = Pool(1, 2, 64, 64, 640)                  # room for the row twice
    x.pool.insert(0, list(range(n)), x.dev(x.k[0]), x.dev(x.v[0]))
    w = sums(x, 1, n)
    if kind == "equal":
        w[:] = 3.5
    elif kind == "one_bit":
        w[:] = (np.float32(1.0).view(np.uint32) + x.rng.integers(0, 2, w.shape).astype(np.uint32)).view(np.float32)
    elif kind == "nan":
        w[:] = np.nan
    was = {0: rows(x, 0)}
    kept, out = x.pool.evict(x.pool.schedule([0], chunk_lists=True), x.dev(w), budget, sink=sink, recent=recent)
    check(x, [0], [0], was, w, budget, sink, recent, kept, out)


@pytest.mark.parametrize("n,H", [(5000, 1), (30_001, 1), (300_000, 2), (450_000, 1)])
def test_weights_in_place_of_long_rows(torch_cuda, n, H):
    """Rows held by one CTA, by several, and (the longest) by none."""
    from prefix_shared_decode_gb300 import Pool
    torch = torch_cuda
    pool = Pool(1, H, 64, 64, -(-n // 64) + 200, n_kv_heads=H)
    k = torch.randn(1, n, H, 64, device="cuda", dtype=torch.float16)
    pool.insert(0, list(range(n)), k, k)
    rows = k[0].cpu().numpy()
    rng = np.random.default_rng(n)
    w = np.round(rng.random((1, 1, H, n + 7)) * 1000).astype(np.float32)        # many ties
    wd = torch.from_numpy(w).cuda()
    mirror = [rows[:, h] for h in range(H)]
    for budget, sink, recent in ((12_000, 5, 9), (4000, 4, 3996)):
        if budget >= n:
            continue
        before = wd.cpu().numpy()
        m = pool.seq_len(0)
        kept, out = pool.evict(pool.schedule([0], chunk_lists=True), wd, budget, sink=sink, recent=recent, out=wd)
        for h in range(H):
            at = OW.kept(before[0, 0, h, :m], budget, sink, recent)
            np.testing.assert_array_equal(kept[0, 0, h].cpu().numpy(), at)
            np.testing.assert_array_equal(wd[0, 0, h, :budget].cpu().numpy(), before[0, 0, h, at])
            assert not wd[0, 0, h, budget:].any()
            mirror[h] = mirror[h][at]
            np.testing.assert_array_equal(pool.read(0)[0][0, :, h].cpu().numpy(), mirror[h])


def test_many_chunks_at_once(torch_cuda):
    """More new chunks than one launch lists."""
    from prefix_shared_decode_gb300 import Pool
    torch = torch_cuda
    x = Cache(torch, 3, "fp16", 16, 64, 1, 1, [300] * 90)
    x.pool = Pool(1, 1, 64, 16, 4000)
    for i in range(90):
        x.pool.insert(i, [1000 * i + j for j in range(300)], x.dev(x.k[i]), x.dev(x.v[i]))
    ids = list(range(90))
    was = {i: rows(x, i) for i in ids}
    w = sums(x, 90, 333)
    kept, out = x.pool.evict(x.pool.schedule(ids, chunk_lists=True), x.dev(w), 200, recent=7)
    check(x, ids, ids, was, w, 200, 0, 7, kept, out)


@pytest.mark.parametrize("kv_dtype,c,D,G,Hkv", [("fp16", 32, 128, 4, 2), ("fp8", 16, 128, 2, 2), ("fp4", 64, 128, 4, 1), ("fp4", 16, 64, 1, 2)])
def test_a_loop_of_steps(torch_cuda, kv_dtype, c, D, G, Hkv):
    """As a serving program does it: steps add up weights, contexts past their
    budget are cut, tokens join, and every call reads what is left."""
    from prefix_shared_decode_gb300 import accumulate_attention, decode_attention, select_chunks, sparse_decode_attention
    torch = torch_cuda
    lens = [9 * c + 5, 4 * c, 7 * c + 1, c - 1]
    x = Cache(torch, 21, kv_dtype, c, D, G, Hkv, lens, L=1, shared=c + 3)
    ids, room, budget, sink, recent = [2, 0, 3, 1], 12 * c, 5 * c + 2, c, 4
    H = G * Hkv
    w = torch.zeros(1, len(ids), Hkv, room, device="cuda")
    sched = x.pool.schedule(ids, chunk_lists=True)
    for round_ in range(3):
        for step in range(3):
            q = x.rng.standard_normal((len(ids), H, D)).astype(np.float16)
            qd = x.dev(q)
            sched = x.pool.schedule(ids, chunk_lists=True, reuse=sched)
            got = decode_attention(x.pool, sched, qd).cpu().numpy()
            accumulate_attention(x.pool, sched, qd, w[0])
            lists = select_chunks(x.pool, sched, qd, 3)
            sparse = sparse_decode_attention(x.pool, sched, qd, lists).cpu().numpy()
            lists = lists.cpu().numpy()
            for r, i in enumerate(ids):
                k, v = (held(t[i][0], kv_dtype, s) for t, s in ((x.k, x.ks), (x.v, x.vs)))
                all_ = [list(range(-(-k.shape[0] // c)))] * Hkv
                for o, chunks in ((got, all_), (sparse, lists[r])):
                    near(o[r], SP.attention(q[r], k, v, chunks, c, D ** -0.5), SP.attention(q[r], k, np.abs(v), chunks, c, D ** -0.5))
            assert sched.device_status() == 0
            for i in ids:
                x.append(i, 1 + (i + step) % 3)
        sched = x.pool.schedule(ids, chunk_lists=True, reuse=sched)
        before = w.cpu().numpy()
        kept, out = x.pool.evict(sched, w, budget, sink=sink, recent=recent, out=w)
        kept = kept.cpu().numpy()
        for r, i in enumerate(ids):
            n = x.k[i].shape[1]
            at = [OW.kept(before[0, r, h, :n], budget, sink, recent) for h in range(Hkv)]
            np.testing.assert_array_equal(kept[0, r, :, :len(at[0])], np.stack(at))
            # the mirror: each head keeps tokens of its own
            x.k[i], x.v[i] = (np.stack([t[0, at[h], h] for h in range(Hkv)], 1)[None] for t in (x.k[i], x.v[i]))
            assert x.pool.seq_len(i) == x.k[i].shape[1] == min(n, budget)


def test_key_bounds_of_the_new_chunks(torch_cuda):
    for kv_dtype, c, D in (("fp16", 16, 64), ("fp8", 32, 128), ("fp4", 16, 128)):
        x = Cache(torch_cuda, 8, kv_dtype, c, D, 1, 2, [10 * c + 3, 6 * c], L=2, ks=0.5)
        w = sums(x, 2, 11 * c)
        kept, _ = x.pool.evict(x.pool.schedule([0, 1], chunk_lists=True), x.dev(w), 3 * c + 4, sink=c, recent=2)
        kept = kept.cpu().numpy()
        for i in range(2):
            for t in (x.k, x.v):
                t[i] = np.stack([np.stack([t[i][l, kept[l, i, h], h] for h in range(2)], 1) for l in range(2)])
        x.check_bounds()
        x.append(0, 5)                    # an append joins the bounds of the last new chunk
        x.check_bounds()


def test_other_streams(torch_cuda):
    """Weights, eviction and a decode in stream order on another stream."""
    from prefix_shared_decode_gb300 import accumulate_attention, decode_attention
    torch = torch_cuda
    x = Cache(torch, 8, "fp16", 32, 128, 2, 2, [700, 300])
    q = x.rng.standard_normal((2, 4, 128)).astype(np.float16)
    qd = x.dev(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        w = torch.zeros(1, 2, 2, 700, device="cuda")
        sched = x.pool.schedule([0, 1], chunk_lists=True)
        accumulate_attention(x.pool, sched, qd, w[0])
        kept, out = x.pool.evict(sched, w, 100, sink=2, recent=2)
        got = decode_attention(x.pool, x.pool.schedule([0, 1]), qd)
    kept2 = kept.cpu().numpy() if side.synchronize() is None else None
    for i in range(2):
        for h in range(2):
            k, v = (held(t[i][0][kept2[0, i, h]], "fp16", 1.0) for t in (x.k, x.v))
            hs = slice(2 * h, 2 * h + 2)
            all_ = [list(range(4))]
            args = (k[:, h:h + 1], v[:, h:h + 1])
            near(got.cpu().numpy()[i, hs], SP.attention(q[i, hs], *args, all_, 32, 128 ** -0.5),
                 SP.attention(q[i, hs], args[0], np.abs(args[1]), all_, 32, 128 ** -0.5))


def test_refusals(torch_cuda):
    from prefix_shared_decode_gb300 import CAError
    torch = torch_cuda
    x = Cache(torch, 8, "fp16", 32, 64, 1, 2, [100, 50])
    sched = x.pool.schedule([0, 1], chunk_lists=True)
    w = torch.zeros(1, 2, 2, 100, device="cuda")
    was = x.pool.stats()
    for bad in (None, w[0], w.double(), w[..., ::2], w.cpu(), w[:, :1], torch.zeros(1, 2, 2, 0, device="cuda")):
        with pytest.raises(ValueError):
            x.pool.evict(sched, bad, 20)
    with pytest.raises(ValueError):
        x.pool.evict(sched, w, 20, out=w[..., :99].contiguous())
    with pytest.raises(CAError, match="INVALID"):
        x.pool.evict(sched, torch.zeros(1, 2, 2, 99, device="cuda"), 20)
    both = torch.zeros(400 + 4, device="cuda")
    with pytest.raises(CAError, match="INVALID"):
        x.pool.evict(sched, both[:400].view(1, 2, 2, 100), 20, out=both[4:].view(1, 2, 2, 100))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    out = torch.empty_like(w)
    with pytest.raises(CAError, match="INVALID"):
        with torch.cuda.graph(graph):
            x.pool.evict(sched, w, 20, out=out)
    assert x.pool.stats() == was
    x.pool.evict(sched, w, 20)
    with pytest.raises(CAError, match="STALE"):
        x.pool.evict(sched, w, 20)


def test_rows_too_long_for_32_bits_are_refused(torch_cuda):
    from prefix_shared_decode_gb300 import capi
    torch = torch_cuda
    x = Cache(torch, 8, "fp16", 32, 64, 1, 2, [100, 50])
    sched = x.pool.schedule([0, 1], chunk_lists=True)
    w, kept = torch.zeros(1, 2, 2, 100, device="cuda"), torch.zeros(1, 2, 2, 20, dtype=torch.int32, device="cuda")
    was = x.pool.stats()
    for room, budget in ((2**31 - 4096, 20), (2**31 - 1, 20), (100, 2**31 - 1)):
        assert capi.lib().ca_evict(x.pool.handle, sched.handle, w.data_ptr(), room, budget, 0, 0, None, kept.data_ptr(),
                                   w.data_ptr(), None) == -9
    assert x.pool.stats() == was
