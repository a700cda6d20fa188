"""How close 8-bit decode attention comes to fp64, with a tolerance for what the kernel does.

Derived, elementwise (u: half a step of the type's rounding):
* A weight, V scale included, is rounded to fp16 for the product with V: 2^-11 of itself, or, below
  fp16's normal range, 2^-25 of the unit.  The unit is at most 2^-7 of the largest weight so far of the warp's
  own tokens (32 of every 128 of a split): groups of tokens are off by 2^-32 n_g max_g (weight) |code|.
* A score is 8 products of 16 dims accumulated in fp32, 2^-23 each of what has been added up: for int8 the
  codes carry a bias of 128, |code + 128| <= 255, which the start of the sum takes out: -128 sum q, itself off
  by 2^-24 for each of its 18 additions.  So off by (8 * 255 * 2 + 18 * 128) 2^-24 sum |q| k_scale scale for
  int8, 8 * 2^-23 sum |q| |code| k_scale scale for e4m3; 1.4427 of that in log2 units, in which the products
  with the scales, log2 of the V scale, the differences to the maxima and the exponentials, those of the
  joins among them (units of O, warps, splits), add 2 * 2^-22 (|x| + 48) + 4 * 2^-21.  The same enters the
  denominator.
* Sums over tokens: a warp adds its share of a split 16 tokens at a time (the sum of weights 4 at a time a
  lane), then 8 lanes, 4 warps and the splits are joined: (split / 32 + 16 + splits) 2^-23 of the terms,
  for numerator and denominator.
* The result is rounded to fp16: 2^-11 of itself, or 2^-25.
"""
import numpy as np
import pytest

import test_gpu_q8 as tq

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def check(got, q, codes, scales, tables, lens, bs, split, code, scale=tq.SCALE, unit=2.0 ** -7):
    S, Hq, _ = q.shape
    Hkv = codes[0].shape[2]
    assert np.isfinite(got).all()
    for s in range(S):
        L = int(lens[s])
        pos = np.arange(L)
        blk, row = tables[s][pos // bs], pos % bs
        group = pos // split * 4 + pos % split // 32 % 4
        for h in range(Hq):
            g = h // (Hq // Hkv)
            K, V = (c[blk, row, g].astype(np.float64) for c in codes)
            ks, vs = (x[blk, g].astype(np.float64) for x in scales)
            qh = q[s, h].astype(np.float64)
            x = scale * (K @ qh) * ks
            p = np.exp(x - x.max())
            p /= p.sum()
            w = p * vs                                       # the weight of a code of V
            ref, spread = w @ V, w @ np.abs(V)
            if code == "int8":
                off = (8 * 255 * 2 + 18 * 128) * 2.0 ** -24 * np.abs(qh).sum() * ks * abs(scale)
            else:
                off = 8 * 2.0 ** -23 * (np.abs(K) @ np.abs(qh)) * ks * abs(scale)
            off = off + 2.0 ** -21 * (np.abs(x) + 48) + 2.0 ** -19   # (nats here, log2 there: 1.4427
            moved = 1.02 * off                                       # ln 2 = 1), of each weight
            mean = (p * moved).sum()                                 # of the denominator
            sums = 2 * (split / 32 + 16 + -(-L // split)) * 2.0 ** -23
            n = np.bincount(group)
            top = np.zeros(len(n))
            np.maximum.at(top, group, w)
            lost = 2.0 ** -25 * unit * (n * top).sum() * np.abs(V).max()
            tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + lost + \
                1.01 * ((w * moved) @ np.abs(V) + (mean + sums + 2.0 ** -11) * spread)
            over = np.abs(got[s, h] - ref) - tol
            assert over.max() <= 0, (s, h, over.max(), tol[over.argmax()])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv", [([100, 2500, 9000], 8, 2), ([5000], 4, 4), ([20000, 1], 8, 1)])
def test_close_to_fp64(ops, code, lens, Hq, Hkv):
    q, codes, scales, tables, lens = tq.decode_case(len(lens) + Hq, lens, Hq, Hkv, 16, code, spread=3)
    scales[0][:] = np.abs(np.random.default_rng(2).standard_normal(scales[0].shape)) * 4 / tq.oq.QMAX[code]
    got, err = tq.run_decode(ops, q, codes, scales, tables, lens, code, 16)
    assert err == 0
    check(got, q, codes, scales, tables, lens, 16,
          ops.split_tokens(len(lens), Hkv, tables.shape[1]), code)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_a_million_tokens(ops, code):
    """Three keys of one weight make up most of the output, in the first, a middle and the last split."""
    long = 2 ** 20 + 7
    q, codes, scales, tables, lens = tq.decode_case(5, [long], 2, 1, 16, code)
    qq = q[0, 0].astype(np.float64)
    for pos in (3, long // 2, long - 1):
        b, r = tables[0, pos // 16], pos % 16
        codes[0][b, r, 0] = tq.oq.nearest_code(qq / np.abs(qq).max() * tq.oq.QMAX[code], code)
        scales[0][b] = 0.5 if code == "int8" else 0.5 / 3.5
    got, err = tq.run_decode(ops, q, codes, scales, tables, lens, code, 16)
    assert err == 0
    check(got, q, codes, scales, tables, lens, 16, ops.split_tokens(1, 1, tables.shape[1]), code)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_small_codes_beside_an_outlier(ops, code, sign):
    """An outlier dim sets a block's scale, the other codes are a few units, and q has one sign: the bias
    of int8 codes, 128 sum q, is far larger than the scores it is taken out of."""
    rng = np.random.default_rng(7)
    lens, Hq, Hkv = [700, 40], 8, 2
    q, codes, scales, tables, lens = tq.decode_case(6, lens, Hq, Hkv, 16, code)
    q = (sign * (1 + rng.uniform(0, 1, q.shape))).astype(np.float16)
    q[..., 11] = 0.001 * sign
    codes[0][:] = rng.integers(-2, 3, codes[0].shape)
    codes[0][..., 11] = tq.oq.QMAX[code] * rng.choice([-1, 1], codes[0].shape[:3])
    scales[0][:] = 0.5
    got, err = tq.run_decode(ops, q, codes, scales, tables, lens, code, 16)
    assert err == 0
    check(got, q, codes, scales, tables, lens, 16, ops.split_tokens(2, Hkv, tables.shape[1]), code)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1)])
def test_many_small_weights_beside_dominant_ones(ops, code, Hq, Hkv):
    """2,000 tokens, one for each warp 25 to 29 log2 units above the others, its V 0 in half of the
    dims: there the others make up the whole output."""
    rng = np.random.default_rng(8)
    q, codes, scales, tables, lens = tq.decode_case(9, [2000], Hq, Hkv, 16, code)
    q[:] = 0
    q[..., 0] = 1
    top = tq.oq.QMAX[code]
    codes[0][:] = 0
    codes[0][..., 0] = tq.oq.nearest_code(-rng.uniform(0.87, 1, codes[0].shape[:3]) * top, code)
    codes[1][:] = tq.oq.nearest_code(rng.uniform(0.5, 1, codes[1].shape) * top, code)
    for warp in range(4):
        b, r = tables[0, 2 * warp], 5
        codes[0][b, r, :, 0] = 0
        codes[1][b, r, :, ::2] = 0
    scales[0][:] = 29 / top
    scales[1][:] = 4000 / top
    got, err = tq.run_decode(ops, q, codes, scales, tables, lens, code, 16, scale=np.log(2))
    assert err == 0
    check(got, q, codes, scales, tables, lens, 16, ops.split_tokens(1, Hkv, tables.shape[1]), code,
          scale=np.log(2))
