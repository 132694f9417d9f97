"""Accumulated attention weights on the GPU, for every pool type, against the
fp64 definition over the stored keys.

Tolerance.  A score is a sum of D products, exact in fp32, in 32 bits: off by at
most (D + 8) 2^-23 times the sum S of their sizes (scale included; a step of
2^-23 for each sum, since the tensor cores may cut instead of rounding).  The
weight exp(x) / sum exp(x) then moves by at most twice that, relatively; its own
exponentials, sum, logarithm and the exponent's rounding (of at most 2^8 in log2
units: 2^-17 absolute) by 2^-15.  The sums of the rows and the running sum add
half a step each."""
import numpy as np
import pytest

from oracle import weights as OW
from tests.test_gpu_sparse import POOLS, Cache, held

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def queries(x, b, q_len, H):
    q = x.rng.standard_normal((b, q_len, H, x.D)).astype(np.float16)
    return q, x.dev(q if q_len > 1 else q[:, 0])


def check(x, ids, q, layer, before, got, scale=None, causal=False):
    """got = before + weights, and before itself past each context."""
    scale = scale or 1 / np.sqrt(x.D)
    G = q.shape[2] // x.Hkv
    before, got = before.astype(np.float64), got.astype(np.float64)
    for r, i in enumerate(ids):
        n = x.k[i].shape[1]
        keys = held(x.k[i][layer], x.kv_dtype, x.ks)
        for h in range(x.Hkv):
            w, size = OW.step_weights(q[r, :, h * G:(h + 1) * G], keys[:, h], scale, causal)
            want = before[r, h, :n] + w
            tol = w * (2 * (x.D + 8) * 2.0**-23 * size + 2.0**-15) + (np.abs(want) + w) * 2.0**-24 * (q.shape[1] * G + 1) + 1e-30
            err = np.abs(got[r, h, :n] - want)
            assert (err <= tol).all(), (i, h, float((err / tol).max()))
            np.testing.assert_array_equal(got[r, h, n:], before[r, h, n:])


@pytest.mark.parametrize("kv_dtype,c,D,G,Hkv", POOLS)
def test_sums_over_steps(torch_cuda, kv_dtype, c, D, G, Hkv):
    """Steps over contexts from one token on with a shared prefix, in place and
    apart, before and after appends that fill partial chunks."""
    from prefix_shared_decode_gb300 import accumulate_attention
    torch = torch_cuda
    lens = [1, c, 5 * c + 3, 17 * c, 40 * c + 7, 3 * c - 1, 33 * c + 1]
    x = Cache(torch, c + D + G, kv_dtype, c, D, G, Hkv, lens, L=2, ks=0.75, vs=1.25, shared=2 * c + 5)
    ids = [4, 0, 2, 6, 1, 5, 3]
    room = 41 * c + 3
    start = x.rng.random((2, len(ids), Hkv, room)).astype(np.float32)
    w = x.dev(start)
    sched = x.pool.schedule(ids)
    for layer in (0, 1):
        q, qd = queries(x, len(ids), 1, Hkv * G)
        assert accumulate_attention(x.pool, sched, qd, w[layer], layer=layer) is not None
        check(x, ids, q, layer, start[layer], w[layer].cpu().numpy())
    # the last chunks grow in place: the same schedule sees the new tokens
    for i in (2, 4, 5, 6):
        x.append(i, 1)
    q, qd = queries(x, len(ids), 1, Hkv * G)
    out = torch.full_like(w[1], -1.0)
    before = w[1].cpu().numpy()
    again = torch.empty_like(out)
    accumulate_attention(x.pool, sched, qd, w[1], out=out, layer=1, scale=0.3)
    accumulate_attention(x.pool, sched, qd, w[1], out=again, layer=1, scale=0.3)
    np.testing.assert_array_equal(w[1].cpu().numpy(), before)
    check(x, ids, q, 1, before, out.cpu().numpy(), scale=0.3)
    assert torch.equal(out, again)
    assert sched.device_status() == 0


@pytest.mark.parametrize("kv_dtype,c,D,G,Hkv,q_len", [("fp16", 16, 64, 2, 2, 3), ("fp16", 64, 128, 4, 2, 4), ("fp16", 32, 256, 2, 1, 16),
                                                      ("fp8", 32, 128, 3, 2, 5), ("fp4", 64, 128, 4, 1, 16), ("fp4", 16, 64, 1, 3, 2)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("no_tpp", [False, True])
def test_several_query_tokens(torch_cuda, kv_dtype, c, D, G, Hkv, q_len, causal, no_tpp):
    from prefix_shared_decode_gb300 import accumulate_attention
    torch = torch_cuda
    lens = [20 * c + 3, q_len, 3 * c + q_len, 9 * c, 20 * c + 1, 20 * c + 2]
    x = Cache(torch, c + q_len, kv_dtype, c, D, G, Hkv, lens, L=1, shared=3 * c)
    ids = [3, 5, 0, 1, 2, 4]
    sched = x.pool.schedule(ids, q_len=q_len, causal=causal, no_tpp=no_tpp)
    q, qd = queries(x, len(ids), q_len, Hkv * G)
    start = np.zeros((len(ids), Hkv, 21 * c), np.float32)
    w = x.dev(start)
    accumulate_attention(x.pool, sched, qd, w)
    check(x, ids, q, 0, start, w.cpu().numpy(), causal=causal)
    assert sched.device_status() == 0


@pytest.mark.parametrize("kv_dtype", ["fp16", "fp8", "fp4"])
def test_one_long_context_and_odd_rooms(torch_cuda, kv_dtype):
    """Many units per context, a room that is the context, and one whose rows
    start off 16 bytes."""
    from prefix_shared_decode_gb300 import accumulate_attention
    x = Cache(torch_cuda, 5, kv_dtype, 16, 128, 4, 2, [20011], L=1)
    sched = x.pool.schedule([0])
    q, qd = queries(x, 1, 1, 8)
    for room in (20011, 20013, 30000):
        w = torch_cuda.ones(1, 2, room, device="cuda")
        accumulate_attention(x.pool, sched, qd, w)
        check(x, [0], q, 0, np.ones((1, 2, room), np.float32), w.cpu().numpy())


def test_scores_of_every_size(torch_cuda):
    """Keys that leave all the weight to one token, and keys that are all alike."""
    from prefix_shared_decode_gb300 import accumulate_attention
    rng = np.random.default_rng(3)
    k = np.zeros((1, 200, 1, 64), np.float16)
    k[0, 77, 0] = 60.0
    k2 = np.ones((1, 130, 1, 64), np.float16) * np.float16(-3.0)
    rows = [(k, k.copy()), (k2, k2.copy())]
    x = Cache(torch_cuda, 5, "fp16", 32, 64, 2, 1, [200, 130], rows=rows)
    q = np.ones((2, 1, 2, 64), np.float16)
    q[:, :, 1] = rng.standard_normal((2, 1, 64)).astype(np.float16)
    w = torch_cuda.zeros(2, 1, 256, device="cuda")
    accumulate_attention(x.pool, x.pool.schedule([0, 1]), x.dev(q[:, 0]), w)
    check(x, [0, 1], q, 0, np.zeros((2, 1, 256), np.float32), w.cpu().numpy())


def test_streams_and_replays(torch_cuda):
    """On another stream; captured, then replayed with other queries and after
    an append; next to a captured decode call, whose workspace stays its own."""
    from prefix_shared_decode_gb300 import accumulate_attention, decode_attention
    torch = torch_cuda
    x = Cache(torch, 9, "fp16", 32, 128, 4, 2, [700, 90, 333], shared=64)
    ids = [2, 0, 1]
    sched = x.pool.schedule(ids)
    q, qd = queries(x, 3, 1, 8)
    side = torch.cuda.Stream()
    w = torch.zeros(3, 2, 800, device="cuda")
    out = torch.empty_like(qd)
    side.wait_stream(torch.cuda.current_stream())
    accumulate_attention(x.pool, sched, qd, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(x, ids, q, 0, np.zeros((3, 2, 800), np.float32), w.cpu().numpy())
    plain = decode_attention(x.pool, sched, qd)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        decode_attention(x.pool, sched, qd, out=out)
        accumulate_attention(x.pool, sched, qd, w)
    for step in range(3):
        if step == 2:
            x.append(0, 3)
        q, new = queries(x, 3, 1, 8)
        qd.copy_(new)
        plain = decode_attention(x.pool, sched, qd)
        before = w.cpu().numpy()
        graph.replay()
        torch.cuda.synchronize()
        check(x, ids, q, 0, before, w.cpu().numpy())
        assert torch.equal(out, plain)
    assert sched.device_status() == 0


def test_a_context_that_outgrows_its_room_is_reported(torch_cuda):
    from prefix_shared_decode_gb300 import accumulate_attention
    torch = torch_cuda
    x = Cache(torch, 9, "fp16", 32, 64, 1, 2, [70, 33])
    sched = x.pool.schedule([0, 1])
    q, qd = queries(x, 2, 1, 2)
    w = torch.zeros(2, 2, 70, device="cuda")
    accumulate_attention(x.pool, sched, qd, w)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        accumulate_attention(x.pool, sched, qd, w)
    graph.replay()
    assert sched.device_status() == 0
    before = w.cpu().numpy()[1]
    x.append(0, 1)
    graph.replay()
    assert sched.device_status() == -7 and sched.device_status() == 0
    got = w.cpu().numpy()
    k = held(x.k[1][0], "fp16", 1.0)
    for h in range(2):                    # the next row was not written into
        want, _ = OW.step_weights(q[1, :, h:h + 1], k[:, h], 1 / 8)
        np.testing.assert_allclose(got[1, h, :33], before[h, :33] + want, rtol=1e-4)


def test_a_wait_that_runs_out_is_reported(torch_cuda):
    from prefix_shared_decode_gb300 import accumulate_attention
    torch = torch_cuda
    for kv_dtype in ("fp16", "fp4"):
        x = Cache(torch, 9, kv_dtype, 32, 128, 4, 2, [300, 200], shared=100)
        sched = x.pool.schedule([0, 1])
        q, qd = queries(x, 2, 1, 8)
        w = torch.zeros(2, 2, 320, device="cuda")
        assert x.pool and __import__("prefix_shared_decode_gb300").capi.lib().ca_sched_inject_stall(sched.handle, 1) == 0
        accumulate_attention(x.pool, sched, qd, w)
        assert sched.device_status() == -8
        w.zero_()
        accumulate_attention(x.pool, sched, qd, w)
        check(x, [0, 1], q, 0, np.zeros((2, 2, 320), np.float32), w.cpu().numpy())
        assert sched.device_status() == 0


def test_refusals(torch_cuda):
    from prefix_shared_decode_gb300 import CAError, accumulate_attention
    torch = torch_cuda
    x = Cache(torch, 9, "fp16", 32, 64, 2, 2, [70, 33])
    sched = x.pool.schedule([0, 1])
    q, qd = queries(x, 2, 1, 4)
    w = torch.zeros(2, 2, 100, device="cuda")
    for bad in (w[:, :1], w.double(), w[..., ::2], w[0], w.cpu(), torch.zeros(2, 2, 0, device="cuda")):
        with pytest.raises(ValueError):
            accumulate_attention(x.pool, sched, qd, bad)
    for bad in (w[..., :99].contiguous(), w.half()):
        with pytest.raises(ValueError):
            accumulate_attention(x.pool, sched, qd, w, out=bad)
    with pytest.raises(ValueError):
        accumulate_attention(x.pool, sched, qd[:1], w)
    with pytest.raises(CAError, match="INVALID"):          # a context of 70 tokens
        accumulate_attention(x.pool, sched, qd, torch.zeros(2, 2, 69, device="cuda"))
    with pytest.raises(CAError, match="INVALID"):
        accumulate_attention(x.pool, sched, qd, w, layer=1)
    both = torch.zeros(2 * 2 * 100 + 4, device="cuda")
    with pytest.raises(CAError, match="INVALID"):          # overlapping, not the same
        accumulate_attention(x.pool, sched, qd, both[:400].view(2, 2, 100), out=both[4:].view(2, 2, 100))
    with pytest.raises(CAError, match="INVALID"):
        accumulate_attention(x.pool, sched, qd, w, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    x.append(0, 64)
    with pytest.raises(CAError, match="STALE"):
        accumulate_attention(x.pool, sched, qd, torch.zeros(2, 2, 200, device="cuda"))
    assert float(w.abs().max()) == 0


@pytest.mark.parametrize("kv_dtype,c,D,G,Hkv", POOLS)
def test_a_query_that_is_no_number_stays_in_its_context(torch_cuda, kv_dtype, c, D, G, Hkv):
    """The sums of its own sequence and head are NaN over the context; those
    behind the context, and every other row's, are as without it."""
    from prefix_shared_decode_gb300 import accumulate_attention
    torch = torch_cuda
    lens, room = [c + 3, 3 * c - 1, 1], 4 * c + 2
    x = Cache(torch, 31, kv_dtype, c, D, G, Hkv, lens)
    sched = x.pool.schedule([0, 1, 2])
    q, qd = queries(x, 3, 1, Hkv * G)
    start = x.rng.random((3, Hkv, room)).astype(np.float32)
    clean, w, apart = x.dev(start), x.dev(start), torch.full((3, Hkv, room), -1.0, device="cuda")
    accumulate_attention(x.pool, sched, qd, clean)
    qd[1, G - 1, 0] = float("nan")                         # of sequence 1 and head 0
    accumulate_attention(x.pool, sched, qd, w.clone(), out=apart)
    accumulate_attention(x.pool, sched, qd, w)
    want = clean.cpu().numpy()
    want[1, 0, :lens[1]] = np.nan
    np.testing.assert_array_equal(w.cpu().numpy(), want)
    np.testing.assert_array_equal(apart.cpu().numpy(), want)


def test_rows_too_long_for_32_bits_are_refused(torch_cuda):
    from prefix_shared_decode_gb300 import capi
    torch = torch_cuda
    x = Cache(torch, 9, "fp16", 32, 64, 2, 2, [70, 33])
    sched = x.pool.schedule([0, 1])
    q, qd = queries(x, 2, 1, 4)
    w, ws = torch.zeros(2, 2, 100, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for room in (2**31 - 4096, 2**31 - 1):
        assert capi.lib().ca_accumulate_attention(x.pool.handle, sched.handle, 0, qd.data_ptr(), w.data_ptr(), w.data_ptr(),
                                                  room, 0.1, ws.data_ptr(), ws.numel(), None) == -9


@pytest.mark.parametrize("kv_dtype,c,D,G,Hkv,q_len", [("fp16", 64, 128, 4, 2, 4), ("fp16", 16, 64, 2, 2, 3), ("fp16", 32, 256, 2, 1, 5),
                                                      ("fp8", 64, 128, 3, 2, 5), ("fp4", 64, 128, 4, 1, 16), ("fp4", 16, 64, 1, 3, 2)])
def test_causal_steps_that_append_in_place(torch_cuda, kv_dtype, c, D, G, Hkv, q_len):
    """Steps that append their tokens and then ask for the schedule again: the mask
    counts from the new ends although no chunk grew.  Sums, and the decode call on
    the same schedule; contexts listed in another order than they lie in the tree."""
    from oracle import cross as OC
    from prefix_shared_decode_gb300 import accumulate_attention, decode_attention
    from tests.test_gpu_fp4 import near
    torch = torch_cuda
    lens = [3 * c + 1, 2 * c + q_len, 5 * c + 2]
    x = Cache(torch, c + q_len, kv_dtype, c, D, G, Hkv, lens, ks=0.75, vs=1.25, shared=2 * c)
    ids = [2, 0, 1]
    w = torch.zeros(3, Hkv, 6 * c, device="cuda")
    sched = None
    for step in range(3):
        if step:
            slots = [x.pool.seq_slots(i) for i in ids]
            x.append(ids[step - 1], min(q_len, c // 4))
            assert [x.pool.seq_slots(i) for i in ids] == slots
        sched = x.pool.schedule(ids, q_len=q_len, causal=True, reuse=sched)
        q, qd = queries(x, 3, q_len, Hkv * G)
        before = w.cpu().numpy()
        accumulate_attention(x.pool, sched, qd, w)
        check(x, ids, q, 0, before, w.cpu().numpy(), causal=True)
        out = decode_attention(x.pool, sched, qd).cpu().numpy()
        for r, i in enumerate(ids):
            k, v = held(x.k[i][0], x.kv_dtype, x.ks), held(x.v[i][0], x.kv_dtype, x.vs)
            near(out[r], OC.attention(q[r], k, v, D ** -0.5, True), OC.attention(q[r], k, np.abs(v), D ** -0.5, True))
    assert sched.device_status() == 0


@pytest.mark.parametrize("room", [96, 99])
def test_sums_behind_the_context_keep_their_bits(torch_cuda, room):
    """In its last chunk and past it, whatever they are: minus zero, infinities, a
    NaN with a payload."""
    from prefix_shared_decode_gb300 import accumulate_attention
    torch = torch_cuda
    x = Cache(torch, 9, "fp16", 32, 64, 2, 2, [70, 33])
    sched = x.pool.schedule([0, 1])
    q, qd = queries(x, 2, 1, 4)
    bits = torch.tensor([-2**31, 0x7f800000, -0x800000, 0x7fc01234, 1, -2**31 + 1], dtype=torch.int32, device="cuda")
    w = bits.repeat(2 * 2 * room // 6 + 1)[:2 * 2 * room].view(2, 2, room).clone()
    w[0, :, :70] = 0
    w[1, :, :33] = 0
    before, sums, out = w.clone(), w.view(torch.float32), torch.full((2, 2, room), 5.0, device="cuda")
    accumulate_attention(x.pool, sched, qd, sums, out=out)
    assert torch.equal(w, before)
    accumulate_attention(x.pool, sched, qd, sums)
    assert torch.equal(out.view(torch.int32), w)
    for r, n in ((0, 70), (1, 33)):
        assert torch.equal(w[r, :, n:], before[r, :, n:])
        assert float((sums[r, :, :n].sum(-1) - 2).abs().max()) < 1e-4      # two query heads a sum
