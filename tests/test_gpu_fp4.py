"""The 4-bit pool on the GPU: stored values bit for bit against the oracle's
quantiser, rows read back from every pool type, and attention over an fp4 pool
through every entry point against the fp64 definition over those values.

Tolerance of an attention output, from its roundings: the fp16 output (half a
step, 2^-11 of the value), the weights p held in fp16 (2^-11 of each, so
2^-11 * A with A = sum p|v| over the softmax), and 2^-12 * A for everything in
32 bits (in units of more than 8 rows the weights' sum is of the rounded ones:
an output then moves by at most 2^-11 * sum p|v - out|; scores: products of fp16 are exact, 128 sums and the scales' fp32
products of magnitude below 2^6 leave below 2^-14 in the exponent; exp2 is
good to 2^-22; weights below fp16's normal range are off by 2^-25 each, 2^-13
over 4096 tokens)."""
import sys

import numpy as np
import pytest

from oracle import attention as A
from oracle import fp4 as F4
from oracle import fp8 as F8
from oracle.pakv import OracleTrie
from tests.treegen import random_segment_sequences

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def rows(rng, L, n, H, D):
    """fp16 rows with sizes that differ by head and a few outliers."""
    x = rng.standard_normal((L, n, H, D)) * np.exp2(rng.integers(-2, 2, (1, 1, H, 1)))
    x[..., int(rng.integers(0, D))] *= 4
    return x.astype(np.float16)


class Cache:
    """An fp4 pool and the oracle's trie over the same sequences."""

    def __init__(self, torch, seed, c, D, G=1, Hkv=2, L=2, k_scale=1.0, v_scale=1.0, n_seqs=12, seqs=None, **kw):
        from prefix_shared_decode_gb300 import Pool
        self.torch, self.rng, self.L, self.Hkv, self.D = torch, np.random.default_rng(seed), L, Hkv, D
        self.ks, self.vs = k_scale, v_scale
        self.seqs = seqs or random_segment_sequences(seed, n_seqs, c, n_segments=10)
        self.pool = Pool(L, Hkv * G, D, c, 900, n_kv_heads=Hkv, kv_dtype="fp4", k_scale=k_scale, v_scale=v_scale, **kw)
        self.trie = OracleTrie(c, 900)
        for i, toks in enumerate(self.seqs):
            k, v = rows(self.rng, L, len(toks), Hkv, D), rows(self.rng, L, len(toks), Hkv, D)
            self.trie.insert(i, toks, F4.roundtrip(k, k_scale), F4.roundtrip(v, v_scale))
            self.pool.insert(i, toks, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())

    def append(self, sid, toks):
        k, v = rows(self.rng, self.L, len(toks), self.Hkv, self.D), rows(self.rng, self.L, len(toks), self.Hkv, self.D)
        self.trie.append(sid, toks, F4.roundtrip(k, self.ks), F4.roundtrip(v, self.vs))
        self.pool.append(sid, toks, self.torch.from_numpy(k).cuda(), self.torch.from_numpy(v).cuda())

    def check_rows(self):
        """Every sequence's rows, read back, are the oracle's values rounded to fp16."""
        ids = list(range(len(self.seqs)))
        k, v = self.pool.read_batch(ids)
        at = 0
        for i in ids:
            n = self.pool.seq_len(i)
            for layer in range(self.L):
                wk, wv = self.trie.materialize(i, layer)
                np.testing.assert_array_equal(k[layer, at:at + n].cpu().numpy(), half(wk))
                np.testing.assert_array_equal(v[layer, at:at + n].cpu().numpy(), half(wv))
            at += n

    def check(self, got, batch, layer, q, scale, causal=False):
        want = (A.decode_attention_multi(self.trie, batch, layer, q, scale, causal) if q.ndim == 4
                else A.decode_attention(self.trie, batch, layer, q, scale))
        near(got, want, weight(self.trie, batch, layer, q, scale, causal))


def half(x):
    """float64 values, rounded to fp32 and then to fp16, as code * scale (exact) times S is."""
    return x.astype(np.float32).astype(np.float16)


def weight(trie, batch, layer, q, scale, causal=False):
    """A = sum p |v| per output element: the definition over |v|."""
    class Abs:
        def materialize(self, s, l):
            k, v = trie.materialize(s, l)
            return k, np.abs(v)
    if q.ndim == 4:
        return A.decode_attention_multi(Abs(), batch, layer, q, scale, causal)
    return A.decode_attention(Abs(), batch, layer, q, scale)


def near(got, want, a):
    got = got.astype(np.float64)
    assert np.isfinite(got).all()
    tol = 2.0 ** -11 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * a + 2.0 ** -25
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, f"error at {worst:.2f} of its bound"


SHAPES = [(16, 64, 1), (32, 64, 4), (64, 64, 1), (16, 128, 1), (32, 128, 1), (64, 128, 1), (64, 128, 4), (32, 128, 8),
          (16, 128, 3), (64, 64, 16), (64, 128, 12)]


@pytest.mark.parametrize("c,D,G", SHAPES)
def test_rows_and_every_output(torch_cuda, c, D, G):
    from prefix_shared_decode_gb300 import decode_attention
    torch = torch_cuda
    x = Cache(torch, 7 + c + D + G, c, D, G, k_scale=0.5, v_scale=0.37)
    x.check_rows()
    batch = [int(i) for i in x.rng.permutation(12)[:10]]
    q = x.rng.standard_normal((10, 2 * G, D)).astype(np.float16)
    qd = torch.from_numpy(q).cuda()
    for layer in range(2):
        for no_tpp in (False, True):
            sched = x.pool.schedule(batch, no_tpp=no_tpp)
            got = decode_attention(x.pool, sched, qd, layer=layer).cpu().numpy()
            assert sched.device_status() == 0
            x.check(got, batch, layer, q, 1 / np.sqrt(D))
    for step, n_add in enumerate((1, 2, c + 3)):            # grow in place, then by chunks
        for sid in batch:
            x.append(sid, [10**6 + 1000 * step + sid * 97 + j for j in range(n_add)])
        x.check_rows()
        sched = x.pool.schedule(batch)
        got = decode_attention(x.pool, sched, qd, layer=1).cpu().numpy()
        assert sched.device_status() == 0
        x.check(got, batch, 1, q, 1 / np.sqrt(D))


@pytest.mark.parametrize("q_len,causal,G,c,D", [(2, False, 1, 16, 64), (4, True, 1, 64, 128), (3, True, 2, 32, 128),
                                               (8, True, 1, 32, 64), (5, True, 4, 64, 128), (16, True, 4, 16, 128),
                                               (3, True, 1, 16, 128), (2, True, 2, 64, 64)])
def test_several_query_tokens(torch_cuda, q_len, causal, G, c, D):
    from prefix_shared_decode_gb300 import decode_attention
    torch = torch_cuda
    x = Cache(torch, 300 + q_len + c, c, D, G)
    batch = [i for i in range(12) if len(x.seqs[i]) >= q_len]
    q = x.rng.standard_normal((len(batch), q_len, 2 * G, D)).astype(np.float16)
    for no_tpp in (False, True):
        sched = x.pool.schedule(batch, no_tpp=no_tpp, q_len=q_len, causal=causal)
        got = decode_attention(x.pool, sched, torch.from_numpy(q).cuda(), layer=1).cpu().numpy()
        assert sched.device_status() == 0
        x.check(got, batch, 1, q, 1 / np.sqrt(D), causal)


@pytest.mark.parametrize("b,shared,own", [(1, 0, 1), (1, 0, 700), (3, 64, 0), (70, 128, 5), (33, 200, 17)])
def test_batches_around_the_tiles(torch_cuda, b, shared, own):
    """One token; one sequence; only shared chunks; more sharers than one
    64-row group; a shared part that ends inside a chunk."""
    from prefix_shared_decode_gb300 import decode_attention
    torch = torch_cuda
    seqs = [list(range(shared)) + [10**6 + 1000 * i + j for j in range(own)] for i in range(b)]
    x = Cache(torch, 11 + b, 64, 128, seqs=seqs, L=1)
    q = x.rng.standard_normal((b, 2, 128)).astype(np.float16)
    sched = x.pool.schedule(list(range(b)))
    got = decode_attention(x.pool, sched, torch.from_numpy(q).cuda()).cpu().numpy()
    assert sched.device_status() == 0
    x.check(got, list(range(b)), 0, q, 1 / np.sqrt(128))


def test_host_buffers_static_scratch_and_graph(torch_cuda, lib):
    from prefix_shared_decode_gb300 import DecodeGraph, decode_attention, decode_attention_host
    torch = torch_cuda
    x = Cache(torch, 21, 64, 128, G=2)
    batch = list(range(12))
    q = x.rng.standard_normal((12, 4, 128)).astype(np.float16)
    qd = torch.from_numpy(q).cuda()
    sched = x.pool.schedule(batch)
    want = decode_attention(x.pool, sched, qd, layer=1)
    x.check(want.cpu().numpy(), batch, 1, q, 1 / np.sqrt(128))
    qh, oh = torch.from_numpy(q).pin_memory(), torch.empty((12, 4, 128), dtype=torch.float16).pin_memory()
    decode_attention_host(x.pool, sched, qh, oh, layer=1)
    torch.cuda.synchronize()
    assert torch.equal(oh, want.cpu())
    out = torch.empty_like(qd)
    assert lib.ca_decode_attention_static_ws(x.pool.handle, sched.handle, 1, qd.data_ptr(), out.data_ptr(),
                                             1 / np.sqrt(128), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, want)
    out.zero_()
    graph = DecodeGraph(x.pool, sched, [(1, qd, out)])
    qd.copy_(torch.from_numpy(-q))
    graph.replay()
    x.check(out.cpu().numpy(), batch, 1, -q, 1 / np.sqrt(128))
    # an append that fits the partial chunks keeps the graph, its quantised row is attended to
    part = [i for i in batch if x.pool.seq_len(i) % 64 not in (0,)]
    for i in part:
        x.append(i, [2 * 10**6 + i])
    graph.replay()
    x.check(out.cpu().numpy(), batch, 1, -q, 1 / np.sqrt(128))


def test_extreme_rows(torch_cuda):
    """Zeros, fp16's largest and smallest values, rows that saturate, ties."""
    from prefix_shared_decode_gb300 import Pool
    torch = torch_cuda
    rng = np.random.default_rng(5)
    n = 50
    k = np.zeros((1, n, 1, 64), np.float16)
    k[0, 1] = 65504
    k[0, 2] = -65504
    k[0, 3] = 2.0 ** -24
    k[0, 4, 0, ::5] = 2.0 ** -14
    k[0, 5] = -0.0
    k[0, 6:30] = rng.choice(np.arange(-48, 49), (24, 1, 64)) / 16           # many ties
    k[0, 30:] = (rng.standard_normal((20, 1, 64)) * np.exp2(rng.integers(-20, 15, (20, 1, 64)))).astype(np.float16)
    v = k[:, ::-1].copy()
    for ks, vs in ((1.0, 1.0), (0.37, 100.0), (2.0 ** -10, 3.0)):
        pool = Pool(1, 1, 64, 16, 10, kv_dtype="fp4", k_scale=ks, v_scale=vs)
        pool.insert(0, list(range(n)), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
        gk, gv = (t.cpu().numpy() for t in pool.read(0))
        np.testing.assert_array_equal(gk, half(F4.roundtrip(k, ks)))
        with np.errstate(over="ignore"):
            np.testing.assert_array_equal(gv, half(F4.roundtrip(v, vs)))


def test_rows_that_are_not_finite_do_no_harm(torch_cuda):
    """A block with an infinity or a NaN keeps finite values, and its
    neighbours' values are theirs."""
    from prefix_shared_decode_gb300 import Pool
    torch = torch_cuda
    rng = np.random.default_rng(6)
    k = rng.standard_normal((1, 20, 1, 64)).astype(np.float16)
    want = half(F4.roundtrip(k, 1.0))
    k[0, 3, 0, 17], k[0, 4, 0, 33], k[0, 5, 0, 0:16] = np.inf, np.nan, np.nan
    pool = Pool(1, 1, 64, 16, 10, kv_dtype="fp4")
    t = torch.from_numpy(k).cuda()
    pool.insert(0, list(range(20)), t, t)
    for got in pool.read(0):
        got = got.cpu().numpy()
        assert np.isfinite(got).all()
        hit = np.zeros((1, 20, 1, 64), bool)
        hit[0, 3, 0, 16:32] = hit[0, 4, 0, 32:48] = hit[0, 5, 0, 0:16] = True
        np.testing.assert_array_equal(got[~hit], want[~hit])


@pytest.mark.parametrize("kv_dtype,c,D", [("fp16", 16, 64), ("fp16", 64, 128), ("fp16", 32, 256), ("fp8", 32, 128),
                                          ("fp8", 64, 128), ("fp4", 16, 128), ("fp4", 64, 64)])
def test_read_ranges_of_every_pool(torch_cuda, kv_dtype, c, D):
    from prefix_shared_decode_gb300 import CAError, Pool
    torch = torch_cuda
    rng = np.random.default_rng(c + D)
    L, H, ks, vs = 2, 3, 0.75, 1.25
    pool = Pool(L, H, D, c, 64, kv_dtype=kv_dtype, k_scale=ks, v_scale=vs)
    lens, held = [1, c, c + 1, 3 * c - 2, 5 * c], {}
    for i, n in enumerate(lens):
        toks = list(range(min(n, 2 * c))) + [1000 * (i + 1) + j for j in range(n - min(n, 2 * c))]
        k, v = rng.standard_normal((2, L, n, H, D)).astype(np.float16)
        m = pool.insert(i, toks, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
        if m:                                                # matched rows are the first inserter's
            src = max(held, key=lambda j: min(held[j][0].shape[1], m))
            k[:, :m], v[:, :m] = held[src][0][:, :m], held[src][1][:, :m]
        held[i] = (k, v)

    def as_held(x, S):
        if kv_dtype == "fp16":
            return x
        return half(F8.dequantize(F8.quantize(x, S), S) if kv_dtype == "fp8" else F4.roundtrip(x, S))

    for ids, starts, ns in ([[4], [0], [5 * c]], [[2, 0, 4, 2], [c, 0, c // 2 + 1, 0], [1, 1, 2 * c, c + 1]],
                            [[3, 1], [2 * c + 1, c], [c - 3, 0]]):
        k, v = pool.read_batch(ids, starts, ns)
        at = 0
        for i, a, n in zip(ids, starts, ns):
            np.testing.assert_array_equal(k[:, at:at + n].cpu().numpy(), as_held(held[i][0][:, a:a + n], ks))
            np.testing.assert_array_equal(v[:, at:at + n].cpu().numpy(), as_held(held[i][1][:, a:a + n], vs))
            at += n
        assert at == k.shape[1]
    # rows behind the last one are left as they were, and another stream may read
    out = [torch.full((L, 2 * c, H, D), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pool.read(4, c, 3 * c, out=out, stream=side)
    side.synchronize()
    assert got[0] is out[0] or got[0].data_ptr() == out[0].data_ptr()
    np.testing.assert_array_equal(out[0].cpu().numpy(), as_held(held[4][0][:, c:3 * c], ks))
    assert pool.read(4, 7, 7)[0].shape[1] == 0
    for bad in (lambda: pool.read(9), lambda: pool.read(0, 0, 2), lambda: pool.read(4, -1, 3),
                lambda: pool.read_batch([9], [0], [0])):
        with pytest.raises(CAError):
            bad()
    for bad in (lambda: pool.read(4, 3, 2), lambda: pool.read_batch([0, 1], [0]),
                lambda: pool.read(4, 0, c, out=(out[0], out[1])),
                lambda: pool.read(4, 0, 2 * c, out=(out[0].cpu(), out[1]))):
        with pytest.raises(ValueError):
            bad()


def test_prompts_longer_than_one_launch(torch_cuda):
    """More chunks than a launch's list holds (1024), all sequences in one call."""
    from prefix_shared_decode_gb300 import Pool
    torch = torch_cuda
    lens = [9000, 1, 8500, 4001]
    total = sum(lens)
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn((1, total, 1, 64), generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    pool = Pool(1, 1, 64, 16, 1400, kv_dtype="fp4")
    pool.insert_batch(list(range(4)), np.arange(total), k, v, lengths=lens)
    gk, gv = pool.read_batch(list(range(4)))
    np.testing.assert_array_equal(gk.cpu().numpy(), half(F4.roundtrip(k.cpu().numpy(), 1.0)))
    np.testing.assert_array_equal(gv.cpu().numpy(), half(F4.roundtrip(v.cpu().numpy(), 1.0)))
    # slots are reused cleanly
    pool.remove_batch([0, 1, 2, 3])
    pool.insert(7, np.arange(100, 8100), k[:, :8000].contiguous(), v[:, :8000].contiguous())
    np.testing.assert_array_equal(pool.read(7)[0].cpu().numpy(), half(F4.roundtrip(k[:, :8000].cpu().numpy(), 1.0)))


def test_offsets_past_32_bits(torch_cuda):
    """A pool of 5.5 GB: the last slots' rows are stored, bounded, read back and
    attended to (whole and by lists) as the first ones'."""
    from prefix_shared_decode_gb300 import Pool, decode_attention, select_chunks, sparse_decode_attention
    torch = torch_cuda
    L, H, D, c, n = 64, 32, 128, 64, 640
    pool = Pool(L, H, D, c, 300, kv_dtype="fp4", chunk_bounds=True)
    g = torch.Generator("cuda").manual_seed(2)
    k, v = (torch.randn((L, n, H, D), generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    for i in range(30):
        pool.insert(i, np.arange(n) + 1000 * i, k, v)
    assert min(pool.seq_slots(29)) * L * H * 9216 > 2 ** 32
    last, first = pool.read(29), pool.read(0)
    assert torch.equal(last[0], first[0]) and torch.equal(last[1], first[1])
    wk, wv = (F4.roundtrip(t[-1].cpu().numpy(), 1.0) for t in (k, v))
    np.testing.assert_array_equal(last[0][-1].cpu().numpy(), half(wk))
    np.testing.assert_array_equal(last[1][-1].cpu().numpy(), half(wv))
    q = torch.randn((2, H, D), generator=g, device="cuda", dtype=torch.float16)
    qn = q.cpu().numpy()
    sched = pool.schedule([29, 3], chunk_lists=True)
    a = np.stack([A.softmax_attention(x, wk, np.abs(wv), D ** -0.5) for x in qn])
    want = np.stack([A.softmax_attention(x, wk, wv, D ** -0.5) for x in qn])
    near(decode_attention(pool, sched, q, layer=L - 1).cpu().numpy(), want, a)
    lists = select_chunks(pool, sched, q, 10, layer=L - 1)
    near(sparse_decode_attention(pool, sched, q, lists, layer=L - 1).cpu().numpy(), want, a)
    hi = torch.from_numpy(wk.reshape(10, c, H, D).max(1)).half()
    assert torch.equal(pool.bounds_view()[pool.seq_slots(29), L - 1, :, 0].cpu(), hi)
    assert sched.device_status() == 0


def test_a_stalled_producer_times_out(torch_cuda, lib):
    """The waits of the fp4 kernel are bounded: a call whose producer never
    issues a copy reports CA_ERR_TIMEOUT, the next one runs."""
    from prefix_shared_decode_gb300 import decode_attention
    torch = torch_cuda
    x = Cache(torch, 17, 16, 64, L=1)
    q = x.rng.standard_normal((12, 2, 64)).astype(np.float16)
    qd = torch.from_numpy(q).cuda()
    sched = x.pool.schedule(list(range(12)))
    assert lib.ca_sched_inject_stall(sched.handle, 1) == 0
    decode_attention(x.pool, sched, qd)
    assert sched.device_status() == -8
    x.check(decode_attention(x.pool, sched, qd).cpu().numpy(), list(range(12)), 0, q, 1 / 8)
    assert sched.device_status() == 0


def test_appends_one_token_at_a_time(torch_cuda):
    """Every place in a chunk, and the first of the next, filled alone: a value
    byte holds two tokens, and the one that was there stays."""
    torch = torch_cuda
    for c, D in ((16, 128), (64, 64)):
        x = Cache(torch, 33 + c, c, D, G=1, Hkv=1, L=2, v_scale=0.5, n_seqs=1, seqs=[list(range(3))])
        for j in range(c + 2):
            x.append(0, [1000 + j])
            if j % 7 == 0 or j > c - 4:
                x.check_rows()
        x.check_rows()


@pytest.mark.parametrize("scale", [128 ** -0.5, -0.05, 0.0, 0.1])
@pytest.mark.parametrize("c,D,G,b", [(64, 128, 1, 70), (16, 64, 3, 21), (32, 128, 20, 3), (64, 64, 40, 2)])
def test_scores_that_rise_along_the_context(torch_cuda, monkeypatch, c, D, G, b, scale):
    """Keys twice as large chunk after chunk, so that a row's softmax reference
    has to follow, in units of 9 to 64 rows; scales of either sign and zero.

    (Scores to base 2: at most 8 steps of mma, each off by at most 16 * 2^-23 of
    its largest term, 0.1 * 1.45 * 8 * 4 * 4 = 18.6 here: 2.9e-4, times ln 2 =
    2.0e-4 of a weight, below the 2^-12 that the bound has for it.)"""
    from prefix_shared_decode_gb300 import decode_attention
    torch = torch_cuda

    def rising(rng, L, n, H, D):
        x = rng.standard_normal((L, n, H, D))
        return (x * np.exp2(np.minimum(np.arange(n) // c, 3))[None, :, None, None]).astype(np.float16)

    monkeypatch.setattr(sys.modules[__name__], "rows", rising)
    seqs = [list(range(6 * c + 5)) + [10**6 + 1000 * i + j for j in range(3 + i % 2 * c)] for i in range(b)]
    x = Cache(torch, 77 + b, c, D, G, seqs=seqs, L=1)
    q = x.rng.standard_normal((b, 2 * G, D)).astype(np.float16)
    sched = x.pool.schedule(list(range(b)))
    got = decode_attention(x.pool, sched, torch.from_numpy(q).cuda(), scale=scale).cpu().numpy()
    assert sched.device_status() == 0
    x.check(got, list(range(b)), 0, q, scale)


@pytest.mark.parametrize("G", [1, 4, 24])
def test_flat_pools_and_a_sequence_twice_in_a_batch(torch_cuda, G):
    """A pool without sharing; a batch that holds one sequence in several rows."""
    from prefix_shared_decode_gb300 import CAError, decode_attention
    torch = torch_cuda
    seqs = [[1000 * i + j for j in range(n)] for i, n in enumerate((1, 200, 64, 33, 513))]
    for kw in (dict(no_sharing=True), {}):
        x = Cache(torch, 91 + G, 32, 128, G, seqs=seqs, **kw)
        x.check_rows()
        for batch in ([4, 1, 0, 3, 2], [1, 4, 1]):
            try:
                sched = x.pool.schedule(batch)
            except CAError as e:
                assert len(set(batch)) < len(batch) and e.name == "CA_ERR_INVALID"
                continue
            q = x.rng.standard_normal((len(batch), 2 * G, 128)).astype(np.float16)
            got = decode_attention(x.pool, sched, torch.from_numpy(q).cuda(), layer=1).cpu().numpy()
            assert sched.device_status() == 0
            x.check(got, batch, 1, q, 1 / np.sqrt(128))
