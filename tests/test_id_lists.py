"""Lists of sequence ids and lengths in every form that the binding takes."""
import numpy as np
import pytest


@pytest.mark.parametrize("form", [list, tuple, lambda x: np.asarray(x, np.int32), np.asarray, lambda x: np.asarray(x, np.uint8),
                                  lambda x: [np.int64(i) for i in x], lambda x: [float(i) for i in x],
                                  lambda x: np.asarray(x, np.float64), lambda x: np.repeat(np.asarray(x), 2)[::2]])
def test_batches_of_any_form(lib, form):
    from prefix_shared_decode_gb300 import CAError, Pool
    p = Pool(1, 2, 64, 16, 40, host_only=True)
    assert p.insert_batch(form([3, 1]), [[1] * 20, [1] * 16 + [2] * 9]) == [0, 16]
    assert p.insert_batch(form([7, 5]), np.arange(40), lengths=form([17, 23])) == [0, 0]
    assert [p.seq_len(i) for i in (1, 3, 5, 7)] == [25, 20, 23, 17]
    with pytest.raises(CAError):
        p.remove_batch(form([1, 9]))
    p.remove_batch(form([5, 1]))
    assert p.stats()["live_seqs"] == 2


def test_lists_that_do_not_go_together(lib):
    from prefix_shared_decode_gb300 import CAError, Pool
    p = Pool(1, 2, 64, 16, 40, host_only=True)
    for bad in (lambda: p.insert_batch([1, 2], np.arange(30), lengths=[20]),
                lambda: p.insert_batch([1, 2], np.arange(30), lengths=[20, 11])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(CAError):
        p.insert_batch([1, 2], np.arange(30), lengths=[20, -1])
    with pytest.raises(CAError):
        p.insert_batch([], [], lengths=[])
    p.remove_batch([])
    assert p.stats()["live_seqs"] == 0
    assert p.insert_batch([1], np.arange(30), lengths=[20, 10]) == [0]      # a length too many is not read
