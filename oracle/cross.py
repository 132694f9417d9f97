"""Attention of query blocks, in fp64 numpy, from its definition."""
import numpy as np


def attention(q, k, v, scale, causal=False):
    """q [m, H, D]; k, v [n, Hkv, D]; with ``causal`` row j sees tokens
    [0, n - m + j], and one that sees none gives zeros."""
    q = np.asarray(q, dtype=np.float64)
    m, H, D = q.shape
    n, HK = k.shape[:2]
    G = H // HK
    out = np.zeros((m, H, v.shape[2]))
    hide = np.arange(n) > n - m + np.arange(m)[:, None]
    for h in range(H):
        x = q[:, h] @ k[:, h // G].T * scale
        if causal:
            x[hide] = -np.inf
        top = x.max(-1, keepdims=True)
        p = np.exp(x - np.where(np.isinf(top), 0.0, top))
        total = p.sum(-1, keepdims=True)
        out[:, h] = (p / np.where(total == 0, 1.0, total)) @ v[:, h // G]
    return out
