"""Decode attention, launch after launch: the same bits every time.

A stage of a ring is read by a warp and then written again by the copy engine.  Were it written
before it has been read, tokens of a later tile would stand in for those of an earlier one, now and
then: two batches that keep the GPU full, one after another, many times.
"""
import numpy as np
import pytest
import torch

import test_gpu_grouped as tg
import test_gpu_q8 as tq
from oracle import attention as oa
from oracle import cache_ops as oc
from parity_helpers import assert_matches_oracle
from paged_kv_cache_138_gb300 import workloads as wl

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


def paged(seed, lens, Hq, Hkv, bs):
    rng = np.random.default_rng([seed, bs])
    nb, tables = tq.batch(rng, lens, bs, pad=-7)
    q = wl.host_normal_fp16(rng, (len(lens), Hq, D))
    kc, vc = (wl.host_normal_fp16(rng, (nb, bs, Hkv, D)) for _ in "kv")
    return q, kc, vc, tables, np.asarray(lens, np.int32)


def check(got, q, kc, vc, tables, lens):
    at = [0, 1, 2, len(lens) - 1]
    assert_matches_oracle(got[at], oa.paged_attention_decode(q[at], kc, vc, tables[at], lens[at], SCALE))


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("bs", [8, 16, 64])
@pytest.mark.parametrize("lens,Hq,Hkv", [([1500] * 60, 8, 8), ([4000, 1, 900, 2047] * 10, 8, 2)])
def test_decode(ops, fused, bs, lens, Hq, Hkv):
    cases = [paged(s, lens, Hq, Hkv, bs) for s in (60, 61)]
    outs, launches = [], []
    for i, (q, kc, vc, tables, lens_) in enumerate(cases):
        out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
        new = [wl.host_normal_fp16(np.random.default_rng([i, n]), (len(lens), Hkv, D)) for n in (0, 1)]
        cache = [dev(kc), dev(vc)]
        if fused:
            launches.append(ops.paged_attention_decode_fused(
                out, dev(q), dev(new[0]), dev(new[1]), *cache, dev(tables), dev(lens_), SCALE,
                prepare=True))
            slots = np.array([oc.slot(tables[s], int(L) - 1, bs) for s, L in enumerate(lens)], np.int64)
            oc.reshape_and_cache(new[0], new[1], slots, kc, vc)
        else:
            launches.append(ops.paged_attention_decode(out, dev(q), *cache, dev(tables), dev(lens_),
                                                       SCALE, prepare=True))
        outs.append(out)
    for got, c in zip(repeat(launches, outs), cases):
        check(got, *c)


@pytest.mark.parametrize("bs", [8, 16, 64])
@pytest.mark.parametrize("Hq,Hkv,groups", [(8, 8, [16, 16, 9]), (32, 8, [4] * 12)])
def test_grouped(ops, bs, Hq, Hkv, groups):
    cases = [tg.forked_case(s, groups, Hq, Hkv, bs, 1536, own_min=1) for s in (70, 71)]
    outs, launches = [], []
    for q, kc, vc, tables, lens in cases:
        gf, sg, gs, mx, mo = ops.shared_prefix_groups(tables, lens, bs, 16 // (Hq // Hkv))
        out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
        launches.append(ops.paged_attention_decode_grouped(
            out, dev(q), dev(kc), dev(vc), dev(tables), dev(lens), dev(gf), dev(sg), dev(gs), mx, mo,
            SCALE, prepare=True))
        outs.append(out)
    for got, c in zip(repeat(launches, outs), cases):
        check(got, *c)
