"""Waits that run out in the two-phase kernel of a 4-bit pool: the call ends,
reports it, and the next call is right."""
import time

import numpy as np
import pytest

from tests.test_gpu_fp4 import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.mark.parametrize("c,D,G,q_len", [(64, 128, 1, 1), (32, 64, 4, 1), (16, 128, 8, 1), (64, 64, 12, 1), (16, 64, 16, 2),
                                         (64, 128, 4, 2), (32, 128, 40, 1)])
def test_waits_that_run_out(torch_cuda, lib, c, D, G, q_len):
    """Units of up to 4, 8, 16, 32 and 64 rows over shared and own chunks.  A
    stalled call's producers copy nothing, and in other CTAs one warp gives up
    at a unit's first tile or inside a head while the others go on: the warps
    meet at a barrier and leave together.

    A call ends within a few limits of about 1 s (the waits of a CTA's warps, its
    producer's turn and its wait for copies in flight): 8 are allowed for."""
    from prefix_shared_decode_gb300 import decode_attention
    torch = torch_cuda
    seqs = [list(range(9 * c + 5)) + [10**6 * (i + 1) + j for j in range(3 + 13 * c * (i % 3))] for i in range(14)]
    x = Cache(torch, 50 + c + G, c, D, G, seqs=seqs, L=1)
    ids = list(range(14))
    shape = (14, 2 * G, D) if q_len == 1 else (14, q_len, 2 * G, D)
    q = x.rng.standard_normal(shape).astype(np.float16)
    qd = torch.from_numpy(q).cuda()
    for no_tpp in (False, True):
        sched = x.pool.schedule(ids, no_tpp=no_tpp, q_len=q_len)
        first = decode_attention(x.pool, sched, qd)
        x.check(first.cpu().numpy(), ids, 0, q, 1 / np.sqrt(D))
        assert sched.device_status() == 0
        assert lib.ca_sched_inject_stall(sched.handle, 1) == 0
        t0 = time.monotonic()
        decode_attention(x.pool, sched, qd)
        assert sched.device_status() == -8
        assert time.monotonic() - t0 < 10
        for _ in range(2):
            assert torch.equal(decode_attention(x.pool, sched, qd), first)
        assert sched.device_status() == 0
