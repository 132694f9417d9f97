"""Attention of query blocks on the GPU, for every pool type, against the fp64
definition over the stored values.

Tolerance of an output: as for the 4-bit pool's attention (tests/
test_gpu_fp4.py): half a step of fp16, the fp16 weights' 2^-11 * A with
A = sum p|v|, and 2^-12 * A for everything held in 32 bits."""
import numpy as np
import pytest

from oracle import cross as OC
from tests.test_gpu_fp4 import near
from tests.test_gpu_sparse import Cache, held

pytestmark = pytest.mark.gpu

POOLS = [("fp16", 16, 64, 1, 2), ("fp16", 64, 64, 3, 2), ("fp16", 32, 64, 8, 1), ("fp16", 64, 128, 4, 2), ("fp16", 16, 128, 1, 3),
         ("fp16", 32, 128, 64, 1), ("fp16", 32, 256, 2, 1), ("fp16", 16, 256, 12, 1), ("fp8", 64, 128, 1, 3),
         ("fp8", 16, 128, 8, 1), ("fp8", 32, 128, 9, 1), ("fp4", 64, 128, 1, 3), ("fp4", 16, 64, 4, 2), ("fp4", 32, 128, 16, 1),
         ("fp4", 64, 64, 3, 2), ("fp4", 16, 128, 5, 1)]


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def queries(x, lens, H):
    q = x.rng.standard_normal((sum(lens), H, x.D)).astype(np.float16)
    return q, x.dev(q)


def check(x, ids, lens, q, layer, got, causal=False, scale=None, n=None):
    got, at = got.cpu().numpy(), 0
    scale = scale or x.D ** -0.5
    for i, m in zip(ids, lens):
        k, v = held(x.k[i][layer], x.kv_dtype, x.ks), held(x.v[i][layer], x.kv_dtype, x.vs)
        mine = q[at:at + m]
        if m:
            near(got[at:at + m], OC.attention(mine, k, v, scale, causal), OC.attention(mine, k, np.abs(v), scale, causal))
        at += m


@pytest.mark.parametrize("kv_dtype,c,D,G,Hkv", POOLS)
@pytest.mark.parametrize("causal", [False, True])
def test_ragged_blocks(torch_cuda, kv_dtype, c, D, G, Hkv, causal):
    """Blocks from no row to several tiles of them, over contexts from one token
    on with a shared prefix; blocks longer than their context, whose first rows
    see nothing under the mask; an id that is listed twice."""
    from prefix_shared_decode_gb300 import cross_attention
    lens = [40 * c + 7, 1, c, 5 * c + 3, 17 * c, 3 * c - 1, 33 * c + 1]
    x = Cache(torch_cuda, c + D + G, kv_dtype, c, D, G, Hkv, lens, L=2, ks=0.75, vs=1.25, shared=2 * c + 5)
    ids = [4, 0, 2, 6, 1, 5, 3, 0]
    blocks = [3, 1, c + 9, 0, 5, 130 // G + 1, 300 // G, 257 // G]
    sched = x.pool.schedule(ids, q_lens=blocks, causal=causal)
    for layer in (1, 0):
        q, qd = queries(x, blocks, G * Hkv)
        out = cross_attention(x.pool, sched, qd, layer=layer)
        check(x, ids, blocks, q, layer, out, causal)
    assert sched.device_status() == 0
    # without the mask the same schedule sees tokens that fill the last chunks
    for i in (3, 5, 6):
        x.append(i, 1)
    if causal:
        sched = x.pool.schedule(ids, q_lens=blocks, causal=True, reuse=sched)
    out = cross_attention(x.pool, sched, qd, layer=1, scale=0.2)
    check(x, ids, blocks, q, 1, out, causal, scale=0.2)
    assert sched.device_status() == 0


@pytest.mark.parametrize("kv_dtype,c,D,G,Hkv", [("fp16", 64, 128, 4, 2), ("fp16", 32, 256, 2, 1), ("fp16", 16, 64, 1, 2),
                                                ("fp8", 64, 128, 4, 1), ("fp4", 64, 128, 2, 2)])
@pytest.mark.parametrize("m,causal", [(1, False), (7, True), (70, True), (600, False)])
def test_long_contexts(torch_cuda, kv_dtype, c, D, G, Hkv, m, causal):
    """Few rows over many chunks: the context is split and joined."""
    from prefix_shared_decode_gb300 import cross_attention
    x = Cache(torch_cuda, m, kv_dtype, c, D, G, Hkv, [9001, 2 * c], ks=0.5)
    blocks = [m, m]
    sched = x.pool.schedule([0, 1], q_lens=blocks, causal=causal)
    q, qd = queries(x, blocks, G * Hkv)
    out = cross_attention(x.pool, sched, qd)
    check(x, [0, 1], blocks, q, 0, out, causal)
    assert torch_cuda.equal(out, cross_attention(x.pool, sched, qd))
    assert sched.device_status() == 0


def test_scores_of_every_size(torch_cuda):
    """Maxima that rise by a little and by a lot from tile to tile, and fall; one
    token with all the weight; keys all alike."""
    from prefix_shared_decode_gb300 import cross_attention
    rng = np.random.default_rng(3)
    rows = []
    for n, size in ((700, np.linspace(-8, 8, 700)), (500, np.linspace(8, -8, 500)), (400, np.where(np.arange(400) == 333, 60.0, 0.0)),
                    (300, np.full(300, -3.0))):
        k = (np.ones((1, n, 1, 64)) * size[None, :, None, None]).astype(np.float16)
        rows.append((k, rng.standard_normal((1, n, 1, 64)).astype(np.float16)))
    x = Cache(torch_cuda, 5, "fp16", 32, 64, 2, 1, [700, 500, 400, 300], rows=rows)
    blocks = [70, 1, 66, 65]
    for causal in (False, True):
        sched = x.pool.schedule([0, 1, 2, 3], q_lens=blocks, causal=causal)
        q = np.ones((sum(blocks), 2, 64), np.float16)
        q[::3] *= np.float16(0.25)
        check(x, [0, 1, 2, 3], blocks, q, 0, cross_attention(x.pool, sched, x.dev(q)), causal)


def test_agrees_with_decode_attention(torch_cuda):
    """A block of a few rows is what the decode call takes for the same queries."""
    from prefix_shared_decode_gb300 import cross_attention, decode_attention
    for causal in (False, True):
        x = Cache(torch_cuda, 5, "fp16", 32, 128, 4, 2, [300, 200, 64], shared=64)
        q, qd = queries(x, [4] * 3, 8)
        a = cross_attention(x.pool, x.pool.schedule([2, 0, 1], q_lens=[4] * 3, causal=causal), qd).float()
        b = decode_attention(x.pool, x.pool.schedule([2, 0, 1], q_len=4, causal=causal), qd.view(3, 4, 8, 128)).float()
        # each is within its tolerance of the same values: |v| weighted is at most 4 here
        assert float((a.view_as(b) - b).abs().max()) <= 2 * 4 * (2.0**-11 + 2.0**-11 + 2.0**-12)


def test_streams_and_replays(torch_cuda):
    from prefix_shared_decode_gb300 import cross_attention
    torch = torch_cuda
    x = Cache(torch, 9, "fp16", 32, 128, 4, 2, [700, 90, 333], shared=64)
    ids, blocks = [2, 0, 1], [70, 9, 200]
    sched = x.pool.schedule(ids, q_lens=blocks)
    q, qd = queries(x, blocks, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = cross_attention(x.pool, sched, qd, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(x, ids, blocks, q, 0, out)
    out = torch.empty_like(qd)
    cross_attention(x.pool, sched, qd, out=out)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    second = torch.empty_like(qd)
    with torch.cuda.graph(graph):
        cross_attention(x.pool, sched, qd, out=out)
        cross_attention(x.pool, sched, out, out=second)
    for step in range(2):
        if step:
            x.append(0, 3)
        q, new = queries(x, blocks, 8)
        qd.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        check(x, ids, blocks, q, 0, out)
        check(x, ids, blocks, out.cpu().numpy(), 0, second)
    assert sched.device_status() == 0


def test_a_prompt_in_its_cache(torch_cuda):
    """A prompt joins behind a prefix that the pool holds: its new tokens attend
    causally, its last queries' weights are added up, the context is cut, and
    decoding goes on over what is left."""
    from prefix_shared_decode_gb300 import accumulate_attention, cross_attention, decode_attention
    from oracle import sparse as SP
    from oracle import weights as OW
    torch = torch_cuda
    for kv_dtype, c, D, G, Hkv in (("fp16", 32, 128, 4, 2), ("fp8", 64, 128, 2, 1), ("fp4", 16, 64, 1, 2)):
        x = Cache(torch, 31, kv_dtype, c, D, G, Hkv, [10 * c + 3, 8 * c + 1], shared=4 * c)
        H, ids = G * Hkv, [1, 0]
        blocks = [4 * c + 1, 6 * c + 3]                     # what is behind the four shared chunks
        q, qd = queries(x, blocks, H)
        out = cross_attention(x.pool, x.pool.schedule(ids, q_lens=blocks, causal=True), qd)
        check(x, ids, blocks, q, 0, out, causal=True)
        # the last four queries of each
        ends = np.cumsum(blocks)
        last = np.stack([q[e - 4:e] for e in ends])
        w = torch.zeros(1, 2, Hkv, 11 * c, device="cuda")
        accumulate_attention(x.pool, x.pool.schedule(ids, q_len=4, causal=True), x.dev(last), w[0])
        sums = w.cpu().numpy()
        sched = x.pool.schedule(ids, chunk_lists=True)
        kept, w = x.pool.evict(sched, w, 5 * c + 2, sink=c, recent=4)
        kept = kept.cpu().numpy()
        q1 = x.rng.standard_normal((2, H, D)).astype(np.float16)
        got = decode_attention(x.pool, x.pool.schedule(ids), x.dev(q1)).cpu().numpy()
        for r, i in enumerate(ids):
            n = x.k[i].shape[1]
            for h in range(Hkv):
                at = OW.kept(sums[0, r, h, :n], 5 * c + 2, c, 4)
                np.testing.assert_array_equal(kept[0, r, h], at)
                k, v = (held(t[i][0][at, h:h + 1], kv_dtype, s) for t, s in ((x.k, x.ks), (x.v, x.vs)))
                hs = slice(h * G, (h + 1) * G)
                all_ = [list(range(6))]
                near(got[r, hs], SP.attention(q1[r, hs], k, v, all_, c, D ** -0.5), SP.attention(q1[r, hs], k, np.abs(v), all_, c, D ** -0.5))


def test_refusals(torch_cuda):
    from prefix_shared_decode_gb300 import CAError, DecodeGraph, accumulate_attention, cross_attention, decode_attention
    from prefix_shared_decode_gb300 import select_chunks
    torch = torch_cuda
    x = Cache(torch, 9, "fp16", 32, 64, 2, 2, [70, 33])
    sched = x.pool.schedule([0, 1], q_lens=[3, 0])
    q, qd = queries(x, [3], 4)
    for bad in (qd[:2], qd.float(), qd[..., ::2], qd.cpu(), qd.view(3, 2, 128)):
        with pytest.raises(ValueError):
            cross_attention(x.pool, sched, bad)
    with pytest.raises(ValueError):
        cross_attention(x.pool, sched, qd, out=qd[:2])
    with pytest.raises(ValueError):
        cross_attention(x.pool, x.pool.schedule([0, 1]), qd)
    with pytest.raises(CAError, match="INVALID"):          # in place
        cross_attention(x.pool, sched, qd, out=qd)
    four = torch.zeros(4, 4, 64, device="cuda", dtype=torch.float16)
    with pytest.raises(CAError, match="INVALID"):          # overlapping by a row
        cross_attention(x.pool, sched, four[:3], out=four[1:])
    with pytest.raises(CAError, match="INVALID"):
        cross_attention(x.pool, sched, qd, layer=1)
    two = torch.zeros(2, 4, 64, device="cuda", dtype=torch.float16)
    for call in (lambda: decode_attention(x.pool, sched, two), lambda: DecodeGraph(x.pool, sched, [(0, two, two.clone())]),
                 lambda: accumulate_attention(x.pool, sched, two, torch.zeros(2, 2, 100, device="cuda")),
                 lambda: sched.plan(), lambda: sched.tables(), lambda: sched.counts()):
        with pytest.raises(CAError, match="INVALID"):
            call()
    for call in (lambda: select_chunks(x.pool, sched, two, 2), lambda: x.pool.evict(sched, torch.zeros(1, 2, 2, 100, device="cuda"), 5)):
        with pytest.raises(ValueError):
            call()
    out = cross_attention(x.pool, sched, qd)
    check(x, [0, 1], [3, 0], q, 0, out)
    none = x.pool.schedule([0, 1], q_lens=[0, 0])
    assert cross_attention(x.pool, none, qd[:0]).shape == (0, 4, 64)
    # one schedule object serves either kind in turn
    sched = x.pool.schedule([0, 1], reuse=sched)
    decode_attention(x.pool, sched, two)
    sched = x.pool.schedule([0, 1], q_lens=[3, 0], reuse=sched)
    assert torch.equal(cross_attention(x.pool, sched, qd), out)
    x.append(0, 64)
    with pytest.raises(CAError, match="STALE"):
        cross_attention(x.pool, sched, qd)


def test_scales_of_every_sign(torch_cuda):
    from prefix_shared_decode_gb300 import cross_attention
    x = Cache(torch_cuda, 13, "fp16", 32, 128, 2, 2, [300, 37])
    blocks = [140, 9]
    for causal in (False, True):
        sched = x.pool.schedule([0, 1], q_lens=blocks, causal=causal)
        q, qd = queries(x, blocks, 4)
        for scale in (-0.1, 0.0, 1e-3):
            out = cross_attention(x.pool, sched, qd, scale=scale).cpu().numpy()
            at = 0
            for i, m in enumerate(blocks):
                k, v = x.k[i][0].astype(np.float64), x.v[i][0].astype(np.float64)
                near(out[at:at + m], OC.attention(q[at:at + m], k, v, scale, causal), OC.attention(q[at:at + m], k, np.abs(v), scale, causal))
                at += m


def test_a_wait_that_runs_out_is_reported(torch_cuda):
    from prefix_shared_decode_gb300 import capi, cross_attention
    x = Cache(torch_cuda, 9, "fp16", 32, 128, 4, 2, [300, 200], shared=100)
    blocks = [100, 50]
    sched = x.pool.schedule([0, 1], q_lens=blocks)
    q, qd = queries(x, blocks, 8)
    assert capi.lib().ca_sched_inject_stall(sched.handle, 1) == 0
    cross_attention(x.pool, sched, qd)
    assert sched.device_status() == -8
    check(x, [0, 1], blocks, q, 0, cross_attention(x.pool, sched, qd))
    assert sched.device_status() == 0


def test_rows_behind_the_last_block_and_unaligned_outputs(torch_cuda):
    """Nothing is written past the blocks' rows; outputs that start 16 bytes off
    a 32-byte boundary."""
    from prefix_shared_decode_gb300 import cross_attention
    torch = torch_cuda
    for kv_dtype, D, G in (("fp16", 64, 3), ("fp16", 128, 4), ("fp8", 128, 2), ("fp16", 256, 2)):
        x = Cache(torch, 17, kv_dtype, 16, D, G, 1, [1500, 77])
        blocks = [131, 6]
        sched = x.pool.schedule([0, 1], q_lens=blocks)
        q, qd = queries(x, blocks, G)
        n = qd.numel()
        room = torch.full((n + 64,), 7.0, device="cuda", dtype=torch.float16)
        for at in (8, 16):
            room.fill_(7.0)
            out = room[at:at + n].view(qd.shape)
            cross_attention(x.pool, sched, qd, out=out)
            check(x, [0, 1], blocks, q, 0, out)
            assert bool((room[:at] == 7).all()) and bool((room[at + n:] == 7).all())


def test_two_schedules_at_once(torch_cuda):
    """Calls on different schedules overlap on two streams."""
    from prefix_shared_decode_gb300 import cross_attention
    torch = torch_cuda
    x = Cache(torch, 23, "fp16", 64, 128, 4, 2, [5000, 3000, 700])
    streams = [torch.cuda.Stream() for _ in range(2)]
    plans = [([0, 2], [70, 300]), ([1, 0], [200, 33])]
    work = []
    for (ids, blocks) in plans:
        sched = x.pool.schedule(ids, q_lens=blocks)
        q, qd = queries(x, blocks, 8)
        work.append((ids, blocks, sched, q, qd, [torch.empty_like(qd) for _ in range(6)]))
    torch.cuda.synchronize()
    for k in range(6):
        for s, (_, _, sched, _, qd, outs) in zip(streams, work):
            cross_attention(x.pool, sched, qd, out=outs[k], stream=s)
    torch.cuda.synchronize()
    for ids, blocks, sched, q, qd, outs in work:
        check(x, ids, blocks, q, 0, outs[0])
        assert all(torch.equal(outs[0], o) for o in outs[1:]) and sched.device_status() == 0


def test_offsets_past_4_gb(torch_cuda):
    """Slots whose tiles lie past 2^32 bytes, for every element size."""
    from prefix_shared_decode_gb300 import Pool, accumulate_attention, cross_attention
    torch = torch_cuda
    for kv_dtype, slots in (("fp16", 9000), ("fp8", 18000), ("fp4", 33000)):
        # 512 KB a slot in fp16: 16 layers of one head of 64 x 128
        pool = Pool(16, 2, 128, 64, slots, n_kv_heads=1, kv_dtype=kv_dtype)
        assert pool._tile_bytes() > 2**32
        g = torch.Generator("cuda").manual_seed(1)
        fill = slots - 12
        row = torch.zeros(16, 1, 1, 128, device="cuda", dtype=torch.float16)
        pool.insert(0, list(range(64 * fill)), row.expand(16, 64 * fill, 1, 128).contiguous(), row.expand(16, 64 * fill, 1, 128).contiguous())
        k, v = (torch.randn(16, 600, 1, 128, device="cuda", dtype=torch.float16, generator=g) for _ in range(2))
        pool.insert(1, [10**8 + j for j in range(600)], k, v)
        pool.remove(0)
        assert min(pool.seq_slots(1)) >= fill
        q = torch.randn(40, 2, 128, device="cuda", dtype=torch.float16, generator=g)
        out = cross_attention(pool, pool.schedule([1], q_lens=[40]), q, layer=15)
        kk, vv = pool.read(1)
        x = torch.einsum("mhd,nd->hmn", q.double(), kk[15, :, 0].double()) / 128**0.5
        p = torch.softmax(x, -1)
        want = torch.einsum("hmn,nd->mhd", p, vv[15, :, 0].double())
        near(out.cpu().numpy(), want.cpu().numpy(), torch.einsum("hmn,nd->mhd", p, vv[15, :, 0].double().abs()).cpu().numpy())
        w = torch.zeros(1, 1, 640, device="cuda")
        accumulate_attention(pool, pool.schedule([1]), q[:1], w, layer=15)
        assert float((w[0, 0, :600].double() - p[:, 0].sum(0)).abs().max()) < 1e-5 and not w[0, 0, 600:].any()
        w = torch.rand(16, 1, 1, 640, device="cuda", generator=g)
        kept, _ = pool.evict(pool.schedule([1], chunk_lists=True), w, 100, sink=3)
        k2, v2 = pool.read(1)
        at = kept[15, 0, 0].long().cpu()
        assert torch.equal(k2[15, :, 0].cpu(), kk[15, :, 0].cpu()[at]) and torch.equal(v2[15, :, 0].cpu(), vv[15, :, 0].cpu()[at])
        del pool, k, v, row


def test_the_call_without_a_workspace_refuses_block_schedules(torch_cuda):
    """Whatever their pieces need; the schedule serves its own call as before."""
    from prefix_shared_decode_gb300 import capi, cross_attention
    torch = torch_cuda
    x = Cache(torch, 9, "fp16", 32, 64, 2, 2, [70, 3000])
    for blocks in ([3, 0], [2, 2]):
        sched = x.pool.schedule([0, 1], q_lens=blocks)
        q, qd = queries(x, blocks, 4)
        four = torch.zeros(4, 4, 64, device="cuda", dtype=torch.float16)
        assert capi.lib().ca_decode_attention_static_ws(x.pool.handle, sched.handle, 0, four.data_ptr(),
                                                        torch.empty_like(four).data_ptr(), 1.0, None) == -1
        check(x, [0, 1], blocks, q, 0, cross_attention(x.pool, sched, qd))


def test_a_refused_build_leaves_the_schedule(torch_cuda):
    """Its calls go on over the tables that were there, masked or not."""
    from prefix_shared_decode_gb300 import CAError, cross_attention
    torch = torch_cuda
    x = Cache(torch, 9, "fp16", 32, 64, 2, 2, [70, 300])
    for causal in (False, True):
        sched = x.pool.schedule([0, 1], q_lens=[300, 4], causal=causal)
        q, qd = queries(x, [300, 4], 4)
        out = cross_attention(x.pool, sched, qd)
        check(x, [0, 1], [300, 4], q, 0, out, causal)
        for ids, lens in (([0, 9], [300, 4]), ([0, 1], [2**31 - 1, 1])):
            with pytest.raises(CAError):
                x.pool.schedule(ids, q_lens=lens, causal=causal, reuse=sched)
            assert torch.equal(cross_attention(x.pool, sched, qd), out)
        assert sched.device_status() == 0
