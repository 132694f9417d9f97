"""A sequence listed twice: a batch has one row per sequence, so a schedule of
it is refused, and so is a removal; nothing changes."""
import numpy as np
import pytest


@pytest.mark.parametrize("no_sharing", [False, True])
def test_repeated_ids_are_refused(lib, no_sharing):
    from prefix_shared_decode_gb300 import CAError, Pool
    p = Pool(1, 2, 64, 16, 60, host_only=True, no_sharing=no_sharing)
    p.insert_batch([1, 4, 6], np.arange(90) % 30, lengths=[30, 40, 20])
    good = p.schedule([4, 1, 6])
    before = good.tables()

    def refused(name, fn):
        with pytest.raises(CAError) as e:
            fn()
        assert e.value.name == name

    for kw in ({}, dict(chunk_lists=True), dict(q_len=4, causal=True), dict(no_tpp=True)):
        refused("CA_ERR_INVALID", lambda: p.schedule([1, 4, 1], **kw))
        refused("CA_ERR_INVALID", lambda: p.schedule([6, 6], **kw))
    refused("CA_ERR_INVALID", lambda: p.remove_batch([1, 1]))
    refused("CA_ERR_EXISTS", lambda: p.insert_batch([9, 9], np.arange(10), lengths=[5, 5]))
    assert p.stats()["live_seqs"] == 3
    again = p.schedule([4, 1, 6]).tables()
    assert all(np.array_equal(before[k], again[k]) for k in before)
