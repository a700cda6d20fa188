"""Prompt attention's host side: the oracle against a loop, and the C entry points'
refusals and workspace sizes (no CUDA call is made)."""
import math

import numpy as np

from oracle import prompt as op


def test_oracle_against_a_loop():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal(s) for s in ((3, 4, 8), (7, 2, 8), (7, 2, 8)))
    out = op.attend(q, k, v, 4, 0.3)[0]
    for i in range(3):
        for h in range(4):
            w = [math.exp(0.3 * float(q[i, h] @ k[t, h // 2])) for t in range(4 + i + 1)]
            ref = sum(a * v[t, h // 2] for t, a in enumerate(w)) / sum(w)
            assert np.abs(out[i, h] - ref).max() < 1e-12
    cache = rng.standard_normal((5, 4, 2, 8))
    got = op.gather(cache, [3, 0], 6)
    assert np.array_equal(got[3], cache[3, 3]) and np.array_equal(got[5], cache[0, 1])


def test_entry_points_refuse_without_a_gpu(native_lib):
    L = native_lib
    p = 4096   # any aligned address: refused before it is used

    def prefill(T=4, S=1, Hq=8, Hkv=2, D=128, bs=16, nb=8, mb=4, q=p, t=p, n=p, qs=p, ws=None, b=0):
        return L.pkv_paged_attention_prefill(p, q, p, p, t, n, qs, T, S, Hq, Hkv, D, bs, nb, mb, 0.1,
                                             ws, b, None, None)

    def packed(T=4, S=1, Hq=8, Hkv=2, D=128, q=p, k=p):
        return L.pkv_prompt_attention(p, q, k, p, p, T, S, Hq, Hkv, D, 0.1, None, None)

    assert prefill(T=0) == 0 and prefill(S=0) == 0 and packed(T=0) == 0 and packed(S=0) == 0
    assert prefill(T=-1) == -1 and prefill(S=-1) == -1 and prefill(Hq=0) == -1
    assert prefill(nb=0) == -1 and prefill(mb=0) == -1 and packed(Hkv=0) == -1
    assert prefill(q=None) == -1 and prefill(t=None) == -1 and prefill(n=None) == -1
    assert prefill(qs=None) == -1 and packed(k=None) == -1
    assert prefill(q=p + 8) == -1 and packed(k=p + 2) == -1
    assert prefill(D=64) == -2 and packed(D=256) == -2
    for bs in (0, 4, 12, 128):
        assert prefill(bs=bs) == -2
    for Hq, Hkv in ((6, 4), (12, 4), (32, 2), (2, 4)):
        assert prefill(Hq=Hq, Hkv=Hkv) == -2 and packed(Hq=Hq, Hkv=Hkv) == -2
    assert prefill(nb=2 ** 31) == -2 and prefill(mb=2 ** 22) == -2 and packed(T=2 ** 26) == -2
    ws = L.pkv_paged_attention_prefill_workspace_bytes
    need = ws(8, 1, 32, 8, 2048, 16)      # 8 rows over 32,768 tokens: the key axis is split
    assert need > 0 and need % (8 * 32 * 130 * 4) == 0
    assert prefill(T=8, Hq=32, Hkv=8, mb=2048, ws=p, b=need - 1) == -1
    assert prefill(T=8, Hq=32, Hkv=8, mb=2048) == -1
    assert prefill(T=8, Hq=32, Hkv=8, mb=2048, ws=p + 8, b=need) == -1
    assert ws(65536, 16, 32, 8, 2048, 16) == 0 and ws(8, 1, 32, 8, 4, 16) == 0
    assert ws(0, 1, 32, 8, 2048, 16) == 0 and ws(8, 1, 12, 4, 2048, 16) == 0
