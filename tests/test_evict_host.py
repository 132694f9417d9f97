"""Eviction's tree: which chunks stay, what the new sequences hold and share, and
that a call which fails changes nothing.  Host-only pools (the choice of tokens
and the rows are tests/test_gpu_evict.py's)."""
import numpy as np
import pytest

ERR = {"INVALID": -1, "OOM": -2, "EXISTS": -4, "STALE": -5}


def make(lib, c=16, cap=200, **kw):
    from prefix_shared_decode_gb300 import Pool
    return Pool(1, 2, 64, c, cap, host_only=True, **kw)


def toks(i, n, shared=0):
    return list(range(shared)) + [10_000 * (i + 1) + j for j in range(n - shared)]


def state(pool, ids, probes=()):
    return (pool.stats(), {i: (pool.seq_slots(i), pool.seq_len(i)) for i in ids}, [pool.match_prefix(t) for t in probes])


def test_in_place(lib):
    pool = make(lib)
    for i, n in enumerate((100, 40, 70)):
        pool.insert(i, toks(i, n, shared=35))
    before = {i: pool.seq_slots(i) for i in range(3)}
    assert pool.stats()["live_slots"] == 2 + 5 + 1 + 3
    sched = pool.schedule([2, 0, 1], chunk_lists=True)
    assert pool.evict(sched, None, 50, sink=20, recent=10) == (None, None)
    # one whole chunk of the sink stays; the rest of 50 tokens take three new chunks, the lowest free slots in batch order
    assert pool.seq_slots(2) == [before[2][0], 11, 12, 13]
    assert pool.seq_slots(0) == [before[0][0], 14, 15, 16]
    assert pool.seq_slots(1) == before[1]
    assert [pool.seq_len(i) for i in range(3)] == [50, 40, 50]
    s = pool.stats()
    assert s["live_slots"] == 1 + 3 + 3 + 2 and s["free_slots"] == 200 - 9 and s["refcount_sum"] == 3 + 3 + 3 + 2
    assert sched.b == 3 and pool.schedule([2, 0, 1], reuse=sched).counts()["b"] == 3
    # the sink still matches, nothing behind it does but what the uncut sequence holds
    assert pool.match_prefix(toks(0, 100, shared=35)) == 32           # sequence 1's second chunk
    pool.remove(1)
    assert pool.match_prefix(toks(0, 100, shared=35)) == 16
    pool.remove(0)
    pool.remove(2)
    assert pool.stats()["free_slots"] == 200 and pool.match_prefix(toks(0, 100, shared=35)) == 0


def test_within_the_budget_nothing_changes(lib):
    pool = make(lib)
    pool.insert(0, toks(0, 40))
    sched = pool.schedule([0], chunk_lists=True)
    was = state(pool, [0])
    pool.evict(sched, None, 40)
    assert state(pool, [0]) == was
    assert pool.evict(sched, None, 100, sink=3, recent=4) == (None, None)     # the schedule is still good
    assert state(pool, [0]) == was


@pytest.mark.parametrize("no_sharing", [False, True])
def test_into_new_sequences(lib, no_sharing):
    pool = make(lib, no_sharing=no_sharing)
    for i, n in enumerate((100, 40, 64)):
        pool.insert(i, toks(i, n, shared=35))
    old = {i: (pool.seq_slots(i), pool.seq_len(i)) for i in range(3)}
    was = pool.stats()
    pool.evict(pool.schedule([0, 1, 2], chunk_lists=True), None, 64, sink=33, into=[70, 71, 72])
    assert {i: (pool.seq_slots(i), pool.seq_len(i)) for i in range(3)} == old
    assert [pool.seq_len(i) for i in (70, 71, 72)] == [64, 40, 64]
    stay = [0, 0, 0] if no_sharing else [2, 2, 4]                # the sink's chunks; every whole chunk of the uncut
    for i in range(3):
        got = pool.seq_slots(70 + i)
        assert got[:stay[i]] == old[i][0][:stay[i]] and len(got) == (4, 3, 4)[i]
        assert not set(got[stay[i]:]) & {x for s, _ in old.values() for x in s}
    assert pool.stats()["live_slots"] == was["live_slots"] + 11 - sum(stay)
    pool.remove_batch([70, 71, 72])
    now = pool.stats()
    assert {k: now[k] for k in now if k != "generation"} == {k: was[k] for k in was if k != "generation"}
    # and the other way round: the old ones leave first
    pool.evict(pool.schedule([0, 1, 2], chunk_lists=True), None, 64, sink=33, into=[70, 71, 72])
    pool.remove_batch([0, 1, 2])
    assert [pool.seq_len(i) for i in (70, 71, 72)] == [64, 40, 64]
    pool.schedule([72, 70, 71]).tables()
    pool.remove_batch([70, 71, 72])
    assert pool.stats()["free_slots"] == 200


def test_what_joins_a_cut_sequence_never_matches(lib):
    """Rows appended behind an eviction were made with tokens that are gone: no
    chunk of theirs may serve a prompt, whether it fills the partial chunk, grows
    behind a new one, or behind a sink that is all that is left."""
    c = 16
    for budget, sink in ((20, 0), (32, 0), (16, 16), (40, 16)):
        pool = make(lib, c)
        prompt = toks(0, 100)
        pool.insert(0, prompt)
        pool.evict(pool.schedule([0], chunk_lists=True), None, budget, sink=sink)
        new = [777_000 + j for j in range(64)]
        for t in new:
            pool.append(0, [t])
        assert pool.seq_len(0) == budget + 64
        for probe in (prompt[:budget] + new, prompt[:sink] + new, new, prompt[:16] + new):
            assert pool.match_prefix(probe) == (c * (sink // c) if probe[:c] == prompt[:c] else 0)
        # copies of a cut sequence are cut too
        pool.evict(pool.schedule([0], chunk_lists=True), None, 1000, into=[5])
        pool.append(5, [888_000 + j for j in range(40)])
        assert pool.match_prefix(prompt[:sink] + new + [888_000 + j for j in range(40)]) == c * (sink // c)


def test_a_copy_of_an_uncut_sequence_matches_as_it_would(lib):
    pool = make(lib)
    pool.insert(0, toks(0, 40))
    pool.evict(pool.schedule([0], chunk_lists=True), None, 40, into=[1])
    pool.remove(0)
    more = [999_000 + j for j in range(30)]
    pool.append(1, more)
    assert pool.match_prefix(toks(0, 40) + more) == 64
    assert pool.insert(2, toks(0, 40) + more) == 64


def test_schedules_over_cut_and_forked_sequences(lib):
    pool = make(lib)
    for i in range(4):
        pool.insert(i, toks(i, 90 + i, shared=50))
    pool.evict(pool.schedule([0, 1], chunk_lists=True), None, 60, sink=32)
    pool.evict(pool.schedule([0, 2, 3], chunk_lists=True), None, 200, into=[10, 12, 13])
    ids = [3, 10, 0, 12, 1, 2, 13]
    t = pool.schedule(ids).tables()
    for p, row in enumerate(t["seq_perm"]):
        own = list(t["sf_chunks"][t["sf_offsets"][p]:t["sf_offsets"][p + 1], 0])
        shared = [int(r[0]) for r in t["cf_rows"] if r[2] <= p < r[3]]
        assert sorted(shared + own) == sorted(pool.seq_slots(ids[row]))


def test_refusals_change_nothing(lib):
    from prefix_shared_decode_gb300 import CAError
    pool = make(lib, cap=12)
    for i in range(2):
        pool.insert(i, toks(i, 90, shared=16))         # 1 + 5 + 5 slots
    lists = pool.schedule([0, 1], chunk_lists=True)
    was = state(pool, [0, 1])
    with pytest.raises(ValueError):
        pool.evict(pool.schedule([0, 1]), None, 20)
    for budget, sink, recent in ((0, 0, 0), (10, 6, 5), (10, -1, 2), (10, 2, -1)):
        with pytest.raises(ValueError):
            pool.evict(lists, None, budget, sink=sink, recent=recent)
    for into in ([5], [5, 6, 7]):
        with pytest.raises(ValueError):
            pool.evict(lists, None, 20, into=into)

    def code(*a, **k):
        with pytest.raises(CAError) as e:
            pool.evict(*a, **k)
        return e.value.code
    assert code(lists, None, 20) == ERR["OOM"]            # four new chunks, one free slot
    assert code(lists, None, 17, sink=16, into=[5, 6]) == ERR["OOM"]
    assert code(lists, None, 16, sink=16, into=[5, 5]) == ERR["INVALID"]
    assert code(lists, None, 16, sink=16, into=[1, 6]) == ERR["EXISTS"]
    assert lib.ca_evict(pool.handle, lists.handle, 8, 100, 20, 0, 0, None, None, None, None) == ERR["INVALID"]
    assert lib.ca_evict(None, lists.handle, None, 0, 20, 0, 0, None, None, None, None) == ERR["INVALID"]
    assert lib.ca_evict(pool.handle, None, None, 0, 20, 0, 0, None, None, None, None) == ERR["INVALID"]
    plain = pool.schedule([0, 1])
    assert lib.ca_evict(pool.handle, plain.handle, None, 0, 20, 0, 0, None, None, None, None) == ERR["INVALID"]
    assert state(pool, [0, 1]) == was
    pool.evict(lists, None, 16, sink=16)                  # needs no new chunk
    assert pool.stats()["live_slots"] == 1 and pool.seq_slots(0) == pool.seq_slots(1)
    assert code(lists, None, 8) == ERR["STALE"]


@pytest.mark.parametrize("fork", [False, True])
def test_a_failed_host_allocation_changes_nothing(lib, fork):
    from prefix_shared_decode_gb300 import CAError
    pool = make(lib)
    for i in range(3):
        pool.insert(i, toks(i, 60 + i, shared=20))
    for i in range(20):                                   # the root keeps an index of its children
        pool.insert(100 + i, toks(100 + i, 5))
    lists = pool.schedule([0, 1, 2], chunk_lists=True)
    probes = [toks(i, 80, shared=20) for i in range(3)]
    ids = list(range(3)) + list(range(100, 120))
    was = state(pool, ids, probes)
    failed = 0
    while True:
        assert lib.ca_pool_inject_alloc_failure(pool.handle, failed) == 0
        try:
            pool.evict(lists, None, 40, sink=5, into=[7, 8, 9] if fork else None)
            break
        except CAError as e:
            assert e.code == ERR["OOM"]
        assert lib.ca_pool_inject_alloc_failure(pool.handle, -1) == 0
        assert state(pool, ids, probes) == was
        failed += 1
    assert lib.ca_pool_inject_alloc_failure(pool.handle, -1) == 0
    assert failed > 8
    # the slots that the failures gave back are taken again in the same order
    fresh = [s for i in ((7, 8, 9) if fork else (0, 1, 2)) for s in pool.seq_slots(i)]
    assert fresh == sorted(fresh) and len(fresh) == 9 and min(fresh) == was[0]["live_slots"]


def test_random_scripts_keep_the_books(lib):
    """Inserts, appends, evictions in place and apart and removes in any order:
    every path's slots are distinct, references add up, and slots come back."""
    rng = np.random.default_rng(11)
    pool = make(lib, cap=400)
    live, nxt = {}, 0
    for step in range(400):
        what = rng.integers(5)
        if what == 0 or len(live) < 2:
            n = int(rng.integers(1, 120))
            pool.insert(nxt, toks(int(rng.integers(4)), n, shared=min(n, int(rng.integers(60)))))
            live[nxt], nxt = n, nxt + 1
        elif what == 1:
            i = int(rng.choice(list(live)))
            k = int(rng.integers(1, 20))
            pool.append(i, [int(x) for x in rng.integers(0, 50, k)])
            live[i] += k
        elif what == 2:
            i = int(rng.choice(list(live)))
            pool.remove(i)
            del live[i]
        else:
            ids = [int(x) for x in rng.permutation(list(live))[:int(rng.integers(1, 4))]]
            sink = int(rng.integers(0, 40))
            budget = sink + int(rng.integers(1, 60))
            into = None if what == 3 else list(range(nxt, nxt + len(ids)))
            pool.evict(pool.schedule(ids, chunk_lists=True), None, budget, sink=sink, into=into)
            for a, b in zip(ids, into or ids):
                live[b] = min(live[a], budget)
            nxt += len(ids) if into else 0
        while len(live) > 12:
            i = next(iter(live))
            pool.remove(i)
            del live[i]
        held, refs = set(), 0
        for i, n in live.items():
            slots = pool.seq_slots(i)
            assert pool.seq_len(i) == n and len(slots) == -(-n // 16) == len(set(slots))
            held |= set(slots)
            refs += len(slots)
        s = pool.stats()
        assert s["live_slots"] == len(held) and s["refcount_sum"] == refs and s["free_slots"] == 400 - len(held)
        pool.schedule(list(live)).tables()
    pool.remove_batch(list(live))
    assert pool.stats()["free_slots"] == 400


def test_a_budget_too_long_for_32_bits_is_refused(lib):
    pool = make(lib, cap=12)
    pool.insert(0, toks(0, 90))
    lists = pool.schedule([0], chunk_lists=True)
    was = state(pool, [0])
    for budget in (2**31 - 4096, 2**31 - 1):
        assert lib.ca_evict(pool.handle, lists.handle, None, 0, budget, 0, 0, None, None, None, None) == -9
    assert lib.ca_evict(pool.handle, lists.handle, None, 2**31 - 1, 20, 0, 0, None, None, None, None) == -9
    assert state(pool, [0]) == was
