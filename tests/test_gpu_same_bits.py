"""Decode attention, launch after launch: the same bits every time.

A stage of a ring is read by a warp and then written again by the copy engine.  Were it written
before it has been read, tokens of a later tile would stand in for those of an earlier one, now and
then: two batches that keep the GPU full, one after another, many times.
"""
import numpy as np
import pytest
import torch

import test_gpu_q8 as tq

pytestmark = pytest.mark.gpu
D = 128
SCALE = 1 / np.sqrt(D)


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


dev = tq.dev


def repeat(launches, outs, times=40):
    """The outputs of the launches' first run; every later one gives the same bits."""
    first = None
    for _ in range(times):
        for out in outs:
            out.fill_(7)
        for _ in range(2):
            for launch in launches:
                launch()
        torch.cuda.synchronize()
        now = [out.clone() for out in outs]
        first = first or now
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(now, first))
    return [out.cpu().numpy() for out in first]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("bs", [8, 16, 64])
@pytest.mark.parametrize("lens,Hq,Hkv", [([1500] * 60, 8, 8), ([4000, 1, 900, 2047] * 10, 8, 2)])
def test_decode_over_8_bit_cache(ops, code, bs, lens, Hq, Hkv):
    cases = [tq.decode_case([s, bs], lens, Hq, Hkv, bs, code) for s in (50, 51)]
    outs, launches = [], []
    for q, codes, scales, tables, lens_ in cases:
        out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
        launches.append(ops.paged_attention_decode_q8(
            out, dev(q), *[tq.codes_to_dev(c, code) for c in codes], *[dev(s) for s in scales],
            dev(tables), dev(lens_), SCALE, prepare=True))
        outs.append(out)
    for got, (q, codes, scales, tables, lens_) in zip(repeat(launches, outs), cases):
        tq.check_decode(got[:4].astype(np.float64), q[:4], codes, scales, tables[:4], lens_[:4], bs)
