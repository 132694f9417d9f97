"""An error that one call reports is that call's alone."""
import ctypes as C

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda(lib):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.mark.parametrize("kv_dtype,bounds", [("fp16", False), ("fp16", True), ("fp8", False), ("fp4", False), ("fp4", True)])
def test_a_failed_call_does_not_fail_the_next(torch_cuda, lib, kv_dtype, bounds):
    """The status word of a schedule cannot be read on a stream that is being
    captured: the call says so, the capture is void, and the inserts, appends and
    reads after it are those of a healthy pool."""
    from prefix_shared_decode_gb300 import Pool
    torch = torch_cuda
    runtime = C.CDLL("libcudart.so.13")          # the one that torch has loaded
    rng = np.random.default_rng(1)
    pool = Pool(1, 2, 128, 16, 40, kv_dtype=kv_dtype, chunk_bounds=bounds)

    def rows(n):
        return torch.from_numpy(rng.standard_normal((1, n, 2, 128)).astype(np.float16)).cuda()

    pool.insert(0, list(range(20)), rows(20), rows(20))
    sched = pool.schedule([0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def fail():
        handle, graph = C.c_void_p(side.cuda_stream), C.c_void_p()
        assert runtime.cudaStreamBeginCapture(handle, 2) == 0              # relaxed: this stream alone
        assert lib.ca_sched_device_status(sched.handle, side.cuda_stream) == -6
        assert runtime.cudaStreamEndCapture(handle, C.byref(graph)) != 0
        runtime.cudaGetLastError()

    k, v = rows(40), rows(40)
    fail()
    assert pool.insert(1, list(range(100, 140)), k, v) == 0
    fail()
    pool.append(1, [7], rows(1), rows(1))
    fail()
    gk, gv = pool.read(1, 0, 40)
    assert pool.seq_len(1) == 41 and sched.device_status() == 0
    if kv_dtype == "fp16":
        assert torch.equal(gk, k) and torch.equal(gv, v)


@pytest.mark.parametrize("chunk_lists", [False, True])
def test_a_schedule_that_fails_keeps_no_memory(torch_cuda, lib, chunk_lists):
    """Its upload is refused on a stream whose capture is void: the buffers it
    had allocated by then (with chunk lists some 4 MB) are given back."""
    from prefix_shared_decode_gb300 import CAError, Pool
    torch = torch_cuda
    runtime = C.CDLL("libcudart.so.13")
    pool = Pool(1, 64, 128, 16, 20000, n_kv_heads=1)
    n = 16 * 15000
    k, v = (torch.zeros((1, n, 1, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    pool.insert(0, np.arange(n), k, v)
    good = pool.schedule([0], chunk_lists=chunk_lists)
    side = torch.cuda.Stream()
    handle, graph = C.c_void_p(side.cuda_stream), C.c_void_p()

    def fail():
        assert runtime.cudaStreamBeginCapture(handle, 2) == 0
        assert lib.ca_sched_device_status(good.handle, side.cuda_stream) == -6
        with pytest.raises(CAError) as e:
            pool.schedule([0], chunk_lists=chunk_lists, stream=side)
        assert e.value.name == "CA_ERR_CUDA"
        assert runtime.cudaStreamEndCapture(handle, C.byref(graph)) != 0
        runtime.cudaGetLastError()

    fail()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(60):
        fail()
    torch.cuda.synchronize()
    lost = free - torch.cuda.mem_get_info()[0]
    assert lost < 8 << 20, f"{lost} bytes"
    assert good.device_status() == 0
    pool.schedule([0], chunk_lists=chunk_lists)
