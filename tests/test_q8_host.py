"""The 8-bit cache's host side: the oracle's codes against their definition, and the
C entry points' refusals (no CUDA call is made)."""
import numpy as np

from oracle import q8 as oq


def test_e4m3_values_and_rounding():
    v = oq.e4m3_bits_to_value(np.arange(256))
    assert v[0x7e] == 448 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0x38] == 1
    assert np.isnan(v[[0x7f, 0xff]]).all()
    values = np.unique(v[np.isfinite(v)])
    y = np.concatenate([np.linspace(-500, 500, 20001), np.geomspace(1e-4, 448, 5000)])
    got = oq.nearest_code(y, "e4m3")
    assert np.isin(got, values).all()
    best = np.abs(values[None] - np.clip(y, -448, 448)[:, None]).min(axis=1)
    assert np.array_equal(np.abs(got - np.clip(y, -448, 448)), best)
    mid = (values[1:] + values[:-1]) / 2     # ties go to the even mantissa
    even = {x for b, x in enumerate(v) if np.isfinite(x) and b % 2 == 0}
    assert all(t in even for t in oq.nearest_code(mid, "e4m3"))
    assert np.array_equal(oq.nearest_code([0.5, 1.5, -2.5, 200], "int8"), [0, 2, -2, 127])


def test_oracle_write_by_hand():
    """Two tokens, then one that doubles the scale: the earlier codes are halved."""
    x = np.zeros((3, 1, 128), np.float16)
    x[0, 0, :2], x[1, 0, 0], x[2, 0, 0] = [127, 3], -20, 254
    codes, scales = np.zeros((2, 8, 1, 128)), np.zeros((2, 4), np.float32)
    t = [[1]]
    oq.write(x[:2], [0, 2], t, [2], codes, scales, 8, "int8")
    assert scales[1, 0] == 1 and list(codes[1, 0, 0, :2]) == [127, 3] and codes[1, 1, 0, 0] == -20
    oq.write(x[2:], [0, 1], t, [3], codes, scales, 8, "int8")
    assert scales[1, 0] == 2 and codes[1, 2, 0, 0] == 127
    assert list(codes[1, 0, 0, :2]) == [64, 2] and codes[1, 1, 0, 0] == -10   # 63.5, 1.5: to even
    assert not codes[0].any() and not codes[1, 3:].any()


def test_entry_points_refuse_without_a_gpu(native_lib):
    L = native_lib
    p = 4096   # any aligned address: refused before it is used

    def write(code=0, T=2, S=1, H=4, D=128, bs=16, nb=8, mb=4, stride=4, k=p, ks=p):
        return L.pkv_reshape_and_cache_q8(k, p, p, p, p, p, p, ks, p, code, T, S, H, D, bs, nb, mb,
                                          stride, None, None)

    def decode(code=0, S=1, Hq=8, Hkv=4, D=128, bs=16, nb=8, mb=4, stride=4, q=p, ks=p, ws=None,
               n=0):
        return L.pkv_paged_attention_decode_q8(p, q, p, p, ks, p, code, p, p, S, Hq, Hkv, D, bs, nb,
                                               mb, stride, 0.1, ws, n, None, None)

    assert write(S=0) == 0 and write(T=0) == 0 and decode(S=0) == 0
    assert write(code=2) == -1 and decode(code=-1) == -1
    assert write(T=-1) == -1 and write(S=-1) == -1 and write(H=0) == -1 and write(nb=0) == -1
    assert write(stride=3) == -1 and decode(stride=3) == -1 and write(mb=0) == -1
    assert write(k=None) == -1 and write(k=p + 8) == -1 and write(ks=p + 2) == -1
    assert write(D=64) == -2 and write(bs=4) == -2 and write(bs=128) == -2
    assert write(nb=2 ** 31) == -2 and write(mb=2 ** 28) == -2
    assert decode(D=64) == -2 and decode(bs=12) == -2 and decode(Hq=12) == -2
    assert decode(Hq=64) == -2 and decode(Hq=6) == -2
    assert decode(q=p + 4) == -1 and decode(q=None) == -1 and decode(ks=None) == -1
    assert decode(S=65536) == -2 and decode(nb=2 ** 31) == -2
    assert decode(mb=64) == -1                                  # needs a workspace
    need = L.pkv_paged_attention_workspace_bytes(1, 8, 64, 16, 128)
    assert need > 0 and decode(mb=64, ws=p, n=need - 1) == -1
    assert decode(mb=64, ws=p + 4, n=need) == -1
