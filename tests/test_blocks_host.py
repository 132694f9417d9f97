"""Schedules of query blocks on host-only pools: what is refused, and reuse."""
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
