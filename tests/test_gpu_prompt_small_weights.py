"""Prompt attention where many tokens of little weight stand beside one that dominates.

Tolerance (derived): as in test_gpu_prompt.py, but a weight below fp16's normal range is off by
2^-25 of the kernel's unit only, and the largest weight is 2^7 units or more: 2^-32 of it.  So n
tokens are off by n 2^-32 of the largest weight; a kernel whose largest weight is 1 unit loses n 2^-25,
2^-9 of the result here.
"""
import math

import numpy as np
import pytest

import test_gpu_prompt as tp
from oracle import prompt as op

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def check_rows(got, q, k, v, rows, scale):
    """The last `rows` rows of a whole prompt."""
    n = k.shape[0]
    ref, spread, peak, mag, vmax = op.attend(q[-rows:], k, v, n - rows, scale)
    x = 1.4427 * mag
    rel = 2.0 ** -11 + 2 * (2.0 ** -20 * x + 2.0 ** -22 * x + 2.0 ** -21) + 2 * (n / 16 + 16) * 2.0 ** -23
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 1.01 * rel[:, :, None] * spread + \
        n * 2.0 ** -32 * (peak * vmax[None])[:, :, None]
    over = np.abs(np.asarray(got[-rows:], np.float64) - ref) - tol
    assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("at", ["first", "middle", "late"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 1)])
def test_many_small_weights_beside_a_dominant_one(ops, at, Hq, Hkv):
    """65,536 tokens, one 25 to 29 log2 units above all others, whose V is 0 in half of the dims:
    there the others make up the whole output."""
    rng = np.random.default_rng(1)
    n = 65536
    q = np.zeros((n, Hq, D), np.float16)
    q[..., 0] = 1
    k, v = np.zeros((n, Hkv, D), np.float16), np.zeros((n, Hkv, D), np.float16)
    k[..., 0] = -rng.uniform(25.1, 29, (n, Hkv))
    v[...] = 1 + rng.uniform(0, 0.5, (n, Hkv, D))
    top = {"first": 0, "middle": n // 2, "late": n - 8}[at]
    k[top, :, 0] = 0
    v[top, :, ::2] = 0
    got, err = tp.run_packed(ops, q, k, v, [0, n], math.log(2))
    assert err == 0
    check_rows(got, q, k, v, 6, math.log(2))


def test_weights_up_to_the_threshold(ops):
    """The running maximum moves only when a score passes it by more than 2^8: keys that lie up to 8
    log2 units above it have the largest weights there are, and keep their fp16 precision."""
    rng = np.random.default_rng(2)
    n = 1024
    q = np.zeros((n, 2, D), np.float16)
    q[..., 0] = 1
    k = np.zeros((n, 2, D), np.float16)
    k[..., 0] = 4
    k[::2, :, 0] = np.float16(11.996)     # tokens are taken from the last tile to the first
    k[896:, :, 0] = 4
    v = rng.choice([-1.0, 1.0], (n, 2, D)).astype(np.float16) * np.float16(60000)
    got, err = tp.run_packed(ops, q, k, v, [0, n], math.log(2))
    assert err == 0
    tp.check(got, q, k, v, 0, math.log(2))
