"""Block tables of a fixed width, far wider than the contexts in them, as a scheduler and a
captured graph have them: the split plan comes from the width, so splits lie past every context,
contexts end in the first split, and rows of one split stand beside rows of several.
Tolerances: those of test_gpu_prompt.py and test_gpu_q8.py.
"""
import numpy as np
import pytest

import test_gpu_prompt as tp
import test_gpu_q8 as tq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def widen(tables, tokens, bs, pad):
    """The table with columns up to `tokens` tokens; what no context reaches is no block."""
    wide = np.full((tables.shape[0], tokens // bs), pad, np.int32)
    wide[:, :tables.shape[1]] = tables
    return wide


@pytest.mark.parametrize("tokens", [32768, 131072, 1 << 20])
@pytest.mark.parametrize("new,cached,Hq,Hkv,bs", [
    ([8, 1, 5], [8184, 4000, 0], 32, 8, 16),
    ([256, 3], [5000, 131], 8, 2, 32),
    ([1, 130, 0, 64], [20000, 900, 50, 64], 8, 1, 8),
])
def test_prefill(ops, tokens, new, cached, Hq, Hkv, bs):
    q, kc, vc, tables, lens = tp.paged_case(sum(new) + bs, new, cached, Hq, Hkv, bs, behind=3)
    wide = widen(tables, tokens, bs, -9)
    assert ops.prefill_workspace_bytes(q.shape[0], len(new), Hq, Hkv, wide.shape[1], bs) > 0
    got, err = tp.run_paged(ops, q, kc, vc, wide, lens, tp.starts(new))
    assert err == 0
    tp.check_paged(got, q, kc, vc, wide, lens, new)
    assert (got[int(np.sum(new)):] == 7).all()


@pytest.mark.parametrize("tokens", [32768, 131072, 1 << 20])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,bs", [(8, 2, 16), (8, 8, 64)])
def test_8bit_decode(ops, tokens, code, Hq, Hkv, bs):
    lens = [1, 0, 511, 513, 2049, 7000]
    q, codes, scales, tables, lens = tq.decode_case(tokens + bs, lens, Hq, Hkv, bs, code)
    wide = widen(tables, tokens, bs, -7)
    got, err = tq.run_decode(ops, q, codes, scales, wide, lens, code, bs)
    assert err == 0 and (got[1] == 0).all()
    tq.check_decode(got, q, codes, scales, wide, lens, bs)
