"""Accumulated attention weights and eviction, in fp64 numpy, from their definitions."""
import numpy as np


def step_weights(q, k, scale, causal=False):
    """What each token of a context is weighed with by a step's queries: q
    [m, G, D] (m query tokens of the group's heads), k [n, D] the stored keys;
    with ``causal`` token j sees k[: n - m + j + 1].  float64 [n], and the
    largest of any row's sum of |q_d k_d| times scale."""
    m, n = q.shape[0], k.shape[0]
    x = np.einsum("jgd,nd->jgn", q.astype(np.float64), k) * scale
    if causal:
        x[np.broadcast_to((np.arange(n) > n - m + np.arange(m)[:, None])[:, None], x.shape)] = -np.inf
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    size = np.einsum("jgd,nd->jgn", np.abs(q.astype(np.float64)), np.abs(k)).max() * scale
    return p.sum((0, 1)), size


def kept(w, budget, sink, recent):
    """Positions that eviction keeps of a context with sums w [n] (float32): the
    first ``sink``, the last ``recent`` and the largest sums between them, ties to
    the lower position, NaN last; ascending, all of a context within its budget."""
    n = len(w)
    if n <= budget:
        return np.arange(n)
    middle = list(range(sink, n - recent))
    middle.sort(key=lambda t: (np.isnan(w[t]), 0.0 if np.isnan(w[t]) else -float(w[t]), t))
    return np.array(sorted(list(range(sink)) + middle[:budget - sink - recent] + list(range(n - recent, n))))
