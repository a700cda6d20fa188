"""TEST INFRASTRUCTURE ONLY: rotary positions in NumPy.

``rotate`` follows the operator's definition, every product and sum rounded to fp32
(NumPy's float32 arithmetic); ``rotate64`` is the same formula in fp64.
"""
import numpy as np


def table64(inv_freq, num_positions, magnitude=1.0):
    angle = np.arange(num_positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    return magnitude * np.stack([np.cos(angle), np.sin(angle)], axis=-1)


def places(query_start, lens, T):
    """(sequence, place in it) of every packed row; -1 where no sequence owns it."""
    seq, place = np.full(T, -1), np.full(T, -1)
    for s, L in enumerate(lens):
        a, b = int(query_start[s]), int(query_start[s + 1])
        seq[a:b], place[a:b] = s, int(L) - (b - a) + np.arange(b - a)
    return seq, place


def _rotate(x, positions, table, axes, adjacent, dtype):
    x = np.asarray(x).astype(dtype)
    table, n = np.asarray(table).astype(dtype), table.shape[1]
    positions = np.atleast_2d(positions)
    y = x.copy()
    for j in range(n):
        at = positions[axes[j] if axes is not None else 0]
        c, s = table[at, j, 0][:, None], table[at, j, 1][:, None]
        i, k = (2 * j, 2 * j + 1) if adjacent else (j, j + n)
        y[..., i] = x[..., i] * c - x[..., k] * s
        y[..., k] = x[..., k] * c + x[..., i] * s
    return y


def rotate(x, positions, table, axes=None, adjacent=False):
    """Rows x [T, H, D] at positions [T] or [axes, T]: fp32, rounded step by step."""
    return _rotate(x, positions, table, axes, adjacent, np.float32)


def rotate64(x, positions, table, axes=None, adjacent=False):
    return _rotate(x, positions, table, axes, adjacent, np.float64)
