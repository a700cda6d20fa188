"""TEST INFRASTRUCTURE ONLY: causal attention of packed prompt rows in fp64 (NumPy)."""
import numpy as np


def attend(q, k, v, first, scale):
    """One sequence: q [n, Hq, D] at positions first .. first + n - 1, k and v [L, Hkv, D].
    Returns the output and, for error bounds: sum of weight * |V| (like out), the
    largest weight and the largest sum of |scale q_i k_i| [n, Hq], the largest |V| [Hq]."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    out, spread = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    peak, mag, vmax = np.zeros((n, Hq)), np.zeros((n, Hq)), np.zeros(Hq)
    see = np.arange(L)[None] <= (first + np.arange(n))[:, None]
    for h in range(Hq):
        g = h // (Hq // Hkv)
        K, V, Q = (np.asarray(a, np.float64) for a in (k[:, g], v[:, g], q[:, h]))
        x = np.where(see, scale * (Q @ K.T), -np.inf)
        p = np.exp(x - x.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        out[:, h], spread[:, h] = p @ V, p @ np.abs(V)
        peak[:, h], vmax[h] = p.max(axis=1), np.abs(V).max()
        mag[:, h] = abs(scale) * np.where(see, np.abs(Q) @ np.abs(K).T, 0).max(axis=1)
    return out, spread, peak, mag, vmax


def gather(cache, table, length):
    """Rows 0 .. length - 1 of a sequence through its block table."""
    bs = cache.shape[1]
    pos = np.arange(length)
    return cache[np.asarray(table)[pos // bs], pos % bs]
