"""Prompt attention of rows whose scores are not finite: the definition's NaN.

A row that sees only scores of -inf (an infinity in its q where the keys have the other sign, or
in the keys it sees) has exp(-inf - -inf), NaN, in every weight; so has a row with a score of
+inf or NaN.  Rows beside it are the same bits as without it.
"""
import numpy as np
import pytest
import torch

import test_gpu_prompt as tp
from paged_kv_cache_138_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


@pytest.mark.parametrize("value", [np.inf, np.nan, -np.inf])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1)])
@pytest.mark.parametrize("n", [1, 100, 128, 300])
def test_packed_query_that_is_not_finite(ops, value, Hq, Hkv, n):
    """Keys of one sign where q is infinite: scores all -inf for +inf, all +inf for -inf."""
    rng = np.random.default_rng(n)
    q = wl.host_normal_fp16(rng, (n + 5, Hq, D))
    k, v = (wl.host_normal_fp16(rng, (n + 5, Hkv, D)) for _ in "kv")
    k[..., 3] = -np.maximum(np.abs(k[..., 3]), np.float16(0.01))
    qs = [0, n, n + 5]
    clean, err = tp.run_packed(ops, q, k, v, qs)
    assert err == 0 and np.isfinite(clean).all()
    for i, h in ((0, 0), (n - 1, Hq - 1), (n // 2, 1)):
        bad = q.copy()
        bad[i, h, 3] = value
        got, err = tp.run_packed(ops, bad, k, v, qs)
        want = clean.copy()
        want[i, h] = np.nan
        assert err == 0 and np.array_equal(got, want, equal_nan=True), (i, h)


@pytest.mark.parametrize("new,cached,Hq,Hkv", [
    ([200, 3], [77, 500], 4, 4),        # units of two tiles; a pair of warpgroups on one
    ([6, 40], [4000, 2500], 8, 2),      # a split key axis
])
def test_paged_query_that_is_not_finite(ops, new, cached, Hq, Hkv):
    q, kc, vc, tables, lens = tp.paged_case(5, new, cached, Hq, Hkv, 16)
    kc[..., 3] = -np.maximum(np.abs(kc[..., 3]), np.float16(0.01))
    clean, err = tp.run_paged(ops, q, kc, vc, tables, lens, tp.starts(new))
    assert err == 0 and np.isfinite(clean).all()
    for i in (0, new[0] - 1, new[0]):
        bad = q.copy()
        bad[i, 1, 3] = np.inf
        got, err = tp.run_paged(ops, bad, kc, vc, tables, lens, tp.starts(new))
        want = clean.copy()
        want[i, 1] = np.nan
        assert err == 0 and np.array_equal(got, want, equal_nan=True), i


def test_first_key_of_minus_infinity(ops):
    """A key that gives -inf: the row that sees nothing else is NaN; for the later ones its weight
    is 0, and they are the definition without it."""
    rng = np.random.default_rng(8)
    n = 140
    q = wl.host_normal_fp16(rng, (n, 2, D))
    q[..., 7] = np.abs(q[..., 7]) + np.float16(0.1)
    k, v = (wl.host_normal_fp16(rng, (n, 2, D)) for _ in "kv")
    k[0, :, 7] = -np.inf
    got, err = tp.run_packed(ops, q, k, v, [0, n])
    assert err == 0 and np.isnan(got[0]).all()
    tp.check(got[1:], q[1:], k[1:], v[1:], 0)
