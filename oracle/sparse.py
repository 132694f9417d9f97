"""Oracle of chunk selection and attention over listed chunks.

TEST INFRASTRUCTURE ONLY (see the package docstring).

bounds: the largest and smallest stored key of each dim over a chunk.
score:  max over the group's query rows of sum_d max(q_d hi_d, q_d lo_d) —
        no token of the chunk has a larger product with the row.
select: all chunks of a context with at most top_k; else its first `sink`
        and last `recent` chunks and the best-scored others, ties to the
        lower number, in ascending order.
"""
from __future__ import annotations

import numpy as np

from .attention import softmax_attention


def bounds(k, c: int) -> np.ndarray:
    """k [n, H, D] -> [chunks, H, 2, D]."""
    k = np.asarray(k, dtype=np.float64)
    parts = [k[a:a + c] for a in range(0, len(k), c)]
    return np.stack([np.stack([p.max(0), p.min(0)], 1) for p in parts])


def scores(q, bnd) -> np.ndarray:
    """q [Hq, D], bnd [chunks, Hkv, 2, D] -> [Hkv, chunks]."""
    q = np.asarray(q, dtype=np.float64)
    HK = bnd.shape[1]
    q = q.reshape(HK, -1, q.shape[-1])
    out = np.empty((HK, len(bnd)))
    for h in range(HK):
        per = np.maximum(q[h][:, None] * bnd[None, :, h, 0], q[h][:, None] * bnd[None, :, h, 1]).sum(-1)
        out[h] = per.max(0)
    return out


def select(score, top_k: int, sink: int, recent: int) -> np.ndarray:
    """score [chunks] of one head -> int [top_k]."""
    n = len(score)
    if n <= top_k:
        return np.concatenate([np.arange(n), np.full(top_k - n, -1)]).astype(np.int64)
    forced = [j for j in range(n) if j < sink or j >= n - recent]
    rest = [j for j in range(n) if sink <= j < n - recent]
    rest.sort(key=lambda j: (-score[j], j))
    return np.array(sorted(forced + rest[:top_k - len(forced)]), dtype=np.int64)


def attention(q, k, v, lists, c: int, scale: float) -> np.ndarray:
    """q [Hq, D]; k, v [n, Hkv, D]; lists[h]: chunk numbers (negative: none)."""
    q, HK = np.asarray(q, dtype=np.float64), k.shape[1]
    G = q.shape[0] // HK
    out = np.zeros(q.shape)
    for h in range(HK):
        at = [t for j in lists[h] if j >= 0 for t in range(j * c, min(len(k), (j + 1) * c))]
        if at:
            out[h * G:(h + 1) * G] = softmax_attention(q[h * G:(h + 1) * G], k[at, h:h + 1], v[at, h:h + 1], scale)
    return out
