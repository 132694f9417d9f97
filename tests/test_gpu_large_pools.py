"""Selection and attention over listed chunks in a pool whose key bounds lie
past 4 GB, with fewer places than chunks: the last slots' bounds are scored,
not those of the slots that 32 bits would reach."""
import numpy as np
import pytest

from oracle import fp4 as F4
from oracle import sparse as SP
from tests.test_gpu_fp4 import near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def test_selection_past_32_bits(torch_cuda):
    from prefix_shared_decode_gb300 import Pool, select_chunks, sparse_decode_attention
    torch = torch_cuda
    L, H, G, D, c, n = 64, 16, 2, 128, 64, 640
    pool = Pool(L, H * G, D, c, 520, n_kv_heads=H, kv_dtype="fp4", chunk_bounds=True)
    g = torch.Generator("cuda").manual_seed(4)

    def rows():
        return torch.randn((L, n, H, D), generator=g, device="cuda", dtype=torch.float16)

    others, k, v = rows(), rows(), rows()
    for i in range(50):
        pool.insert(i, np.arange(n) + 1000 * i, others, others)
    pool.insert(50, np.arange(n) + 10**6, k, v)
    assert min(pool.seq_slots(50)) * L * H * 9216 > 2 ** 32
    assert pool.bounds_view().storage_offset() * 2 > 2 ** 32
    layer = L - 1
    held = [F4.roundtrip(t[layer].cpu().numpy(), 1.0) for t in (k, v)]
    bounds = SP.bounds(held[0], c)
    got = pool.bounds_view()[pool.seq_slots(50), layer].cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(got, bounds)
    q = torch.randn((2, H * G, D), generator=g, device="cuda", dtype=torch.float16)
    qn = q.cpu().numpy()
    sched = pool.schedule([7, 50], chunk_lists=True)
    for top_k, sink, recent in ((1, 0, 0), (4, 1, 1), (7, 0, 2), (9, 2, 0)):
        lists = select_chunks(pool, sched, q, top_k, layer=layer, sink=sink, recent=recent)
        want = np.stack([SP.select(s, top_k, sink, recent) for s in SP.scores(qn[1], bounds)])
        np.testing.assert_array_equal(lists[1].cpu().numpy(), want)
        out = sparse_decode_attention(pool, sched, q, lists, layer=layer)[1].cpu().numpy()
        near(out, SP.attention(qn[1], *held, want, c, D ** -0.5),
             SP.attention(qn[1], held[0], np.abs(held[1]), want, c, D ** -0.5))
    assert sched.device_status() == 0
