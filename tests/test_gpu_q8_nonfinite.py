"""8-bit decode attention of queries and scales that are not finite: NaN, and only where it belongs.

An infinity or NaN in one head's q makes every score of that head infinite or NaN, so its softmax
and its whole output row are NaN, by the definition (exp(inf - inf), and for scores that are all
-inf exp(-inf - -inf)); so does a NaN or infinite scale, for every head.  Zeros would look like a
healthy layer.  Heads and sequences beside it are computed apart from it: the same bits as without.
A context of no tokens gives zeros whatever q holds.
"""
import numpy as np
import pytest
import torch

import test_gpu_q8 as tq

pytestmark = pytest.mark.gpu
SCALE = tq.SCALE


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


# the longest context: 1 split, 2 to 7 (merged by a warp a row), 8 and more (by a CTA a row)
LONGEST = [300, 1000, 3584, 8700]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("longest", LONGEST)
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (8, 1)])
def test_query_that_is_not_finite(ops, code, longest, Hq, Hkv):
    lens = [70, longest, 0, longest // 2]
    q, codes, scales, tables, lens = tq.decode_case(longest + Hq, lens, Hq, Hkv, 16, code)
    clean, err = tq.run_decode(ops, q, codes, scales, tables, lens, code, 16)
    assert err == 0 and np.isfinite(clean).all()
    for value in (np.nan, np.inf, -np.inf):
        for s, h in ((1, 2), (3, Hq - 1), (2, 0)):
            bad = q.copy()
            bad[s, h, 17] = value
            got, err = tq.run_decode(ops, bad, codes, scales, tables, lens, code, 16)
            want = clean.copy()
            if lens[s]:
                want[s, h] = np.nan
            assert err == 0 and np.array_equal(got, want, equal_nan=True), (value, s, h)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("longest", LONGEST)
def test_scores_that_are_all_minus_infinity(ops, code, longest):
    """An infinity in q where every key has the other sign: not a head without tokens."""
    q, codes, scales, tables, lens = tq.decode_case(longest, [longest, 33], 8, 2, 16, code)
    codes[0][..., 5] = -np.maximum(np.abs(codes[0][..., 5]), 1)
    clean, _ = tq.run_decode(ops, q, codes, scales, tables, lens, code, 16)
    q[0, 6, 5] = np.inf
    got, err = tq.run_decode(ops, q, codes, scales, tables, lens, code, 16)
    clean[0, 6] = np.nan
    assert err == 0 and np.array_equal(got, clean, equal_nan=True)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("longest", LONGEST)
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_scale_that_is_not_finite(ops, code, longest, scale):
    q, codes, scales, tables, lens = tq.decode_case(longest, [longest, 0, 33], 8, 2, 16, code)
    got, err = tq.run_decode(ops, q, codes, scales, tables, lens, code, 16, scale=scale)
    assert err == 0
    assert np.isnan(got[[0, 2]]).all() and (got[1] == 0).all()


def test_one_split_of_many(ops):
    """The NaN meets the other splits in the merge: a key of NaN code in one block of a long
    context makes the heads that read it NaN, and no others."""
    q, codes, scales, tables, lens = tq.decode_case(3, [6000, 6000], 8, 2, 16, "e4m3")
    clean, _ = tq.run_decode(ops, q, codes, scales, tables, lens, "e4m3", 16)
    codes[0][tables[0, 200], 3, 1, 9] = np.nan
    got, err = tq.run_decode(ops, q, codes, scales, tables, lens, "e4m3", 16)
    clean[0, 4:] = np.nan
    assert err == 0 and np.array_equal(got, clean, equal_nan=True)
