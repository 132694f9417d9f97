"""Schedules of query blocks on host-only pools: what is refused, and reuse."""
import ctypes as C
import os
import shutil
import subprocess

import pytest


def make(lib):
    from prefix_shared_decode_gb300 import Pool
    pool = Pool(1, 4, 64, 16, 100, host_only=True, n_kv_heads=2)
    pool.insert(0, list(range(100)))
    pool.insert(1, list(range(40)))
    return pool


def test_refusals(lib):
    from prefix_shared_decode_gb300 import CAError, cross_attention
    pool = make(lib)
    sched = pool.schedule([1, 0, 1], q_lens=[5, 0, 7], causal=True)
    assert sched.q_lens == [5, 0, 7] and sched.b == 3 and sched.device_status() == 0
    for kw in (dict(q_len=2), dict(no_tpp=True), dict(chunk_lists=True)):
        with pytest.raises(ValueError):
            pool.schedule([0, 1], q_lens=[1, 1], **kw)
    for lens in ([1], [1, 2, 3], [1, -1]):
        with pytest.raises(ValueError):
            pool.schedule([0, 1], q_lens=lens)
    with pytest.raises(CAError, match="NOT_FOUND"):
        pool.schedule([0, 7], q_lens=[1, 1])
    with pytest.raises(CAError, match="INVALID"):
        pool.schedule([], q_lens=[])
    with pytest.raises(CAError, match="UNSUPPORTED"):
        pool.schedule([0, 1], q_lens=[2**31 - 1, 1])
    for call in (sched.tables, sched.counts, sched.plan):
        with pytest.raises(CAError, match="INVALID"):
            call()
    with pytest.raises(ValueError):
        cross_attention(pool, sched, None)
    assert lib.ca_cross_attention(pool.handle, sched.handle, 0, None, None, 1.0, None, 0, None) == -1
    assert lib.ca_build_schedule_blocks(None, None, 1, None, 0, None, None) == -1


def test_reuse(lib):
    pool = make(lib)
    sched = pool.schedule([0, 1], q_lens=[300, 4])
    key, need = sched._key(), sched.workspace_bytes()
    assert pool.schedule([0, 1], q_lens=[300, 4], reuse=sched)._key() == key
    assert pool.schedule([0, 1], q_lens=[300, 5], reuse=sched)._key() != key
    # either kind in turn
    assert pool.schedule([0, 1], reuse=sched).counts()["b"] == 2
    assert pool.schedule([0, 1], q_lens=[300, 4], reuse=sched).workspace_bytes() == need
    # a failed build leaves the tables that were there
    with pytest.raises(Exception):
        pool.schedule([0, 9], q_lens=[300, 4], reuse=sched)
    assert sched._key() == key and sched.workspace_bytes() == need


STATIC_WS = r"""
// A schedule of query blocks handed to ca_decode_attention_static_ws: the pool and
// the schedule are made to look like a device's, which nothing reads before the
// call's checks are through.
#include "ca_internal.h"
#include <cstdio>
int main() {
    const ca_pool_config cfg{1, 4, 64, 16, 100, 0u};
    ca_pool* pool = nullptr;
    ca_sched* sched[2] = {nullptr, nullptr};
    int32_t tokens[40], m = 3;
    const int64_t id = 0;
    for (int i = 0; i < 40; ++i) tokens[i] = i;
    if (ca_pool_create(&cfg, nullptr, 0, &pool) || ca_insert_tokens(pool, 0, tokens, 40, nullptr, nullptr, nullptr, nullptr) ||
        ca_build_schedule_blocks(pool, &id, 1, &m, 0, &sched[0], nullptr) || ca_build_schedule(pool, &id, 1, &sched[1], nullptr))
        return 2;
    alignas(1024) static unsigned char bytes[1024];
    reinterpret_cast<ca::Pool*>(pool)->kv = bytes;
    reinterpret_cast<ca::Pool*>(pool)->device = -1;     // no device: the call ends there at the latest
    for (ca_sched* s : sched) {
        reinterpret_cast<ca::Sched*>(s)->dev = bytes;
        std::printf("%d %d\n", ca_decode_attention_static_ws(pool, s, 0, bytes, bytes + 512, 1.f, nullptr),
                    ca_decode_attention_static_ws(pool, s, 1, bytes, bytes + 512, 1.f, nullptr));
    }
}
"""


def test_the_call_without_a_workspace_refuses_them(lib, tmp_path):
    from prefix_shared_decode_gb300 import build, capi
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "static_ws.cpp", tmp_path / "static_ws"
    src.write_text(STATIC_WS)
    subprocess.run([cxx, "-std=c++17", f"-I{build.CSRC}", f"-I{build._cuda_home()}/include", str(src), "-o", str(exe),
                    capi.LIB_PATH, f"-Wl,-rpath,{os.path.dirname(capi.LIB_PATH)}"], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, (run.returncode, run.stderr)
    blocks, plain = (line.split() for line in run.stdout.splitlines())
    assert blocks == ["-1", "-1"]
    assert plain[0] in ("-1", "-6") and plain[1] == "-1"     # no such device, or none at all


def test_the_other_calls_workspaces_are_refused(lib):
    pool = make(lib)
    n = C.c_size_t(7)
    for kw in (dict(q_lens=[300, 4]), dict()):
        sched = pool.schedule([0, 1], **kw)
        for call in (lib.ca_workspace_bytes_host, lib.ca_workspace_bytes_weights):
            assert call(sched.handle, C.byref(n)) == (-1 if kw else 0)
        assert lib.ca_workspace_bytes(sched.handle, C.byref(n)) == 0


def test_sizes_past_32_bits_are_refused(lib):
    """Before anything is built over them: the last case has 42 million tiles."""
    import resource
    from prefix_shared_decode_gb300 import CAError, Pool
    pools = {}
    for G, D, T in ((64, 128, 256), (32, 256, 128), (1, 64, 256)):
        pools[G] = pool = Pool(1, G, D, 16, 20, host_only=True, n_kv_heads=1)
        pool.insert(0, list(range(100)))
        most = (2**31 - 1 - T) // G
        before = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss
        for lens in ([most + 1], [3, most + 1], [2**31 - 1], [most] * 65):
            with pytest.raises(CAError, match="UNSUPPORTED"):
                pool.schedule([0] * len(lens), q_lens=lens)
        assert resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - before < 64 * 1024      # KB
    most = (2**31 - 1 - 256) // 64
    before = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss
    with pytest.raises(CAError, match="UNSUPPORTED"):
        pools[64].schedule([0] * 5, q_lens=[most] * 5)
    assert resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - before < 64 * 1024
