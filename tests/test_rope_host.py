"""Rotary positions on the host: the oracle against a loop and complex numbers, tables and
sections, the C entry points' refusals (no CUDA call is made) and the wrappers' (stand-ins
for CUDA tensors and a library that only records)."""
import math

import numpy as np
import pytest
import torch

from oracle import rope as orope
from paged_kv_cache_138_gb300 import ops as real_ops

F16, F32, I32 = torch.float16, torch.float32, torch.int32


@pytest.mark.parametrize("adjacent", [False, True])
def test_oracle_is_a_rotation(adjacent):
    rng = np.random.default_rng(1)
    n, D = 3, 8
    table = orope.table64([1.0, 0.3, 0.01], 50)
    x, pos = rng.standard_normal((4, 2, D)), np.array([[0, 7, 49, 3], [1, 2, 30, 3]])
    axes = (0, 1, 0)
    y = orope.rotate64(x, pos, table, axes, adjacent)
    for t in range(4):
        for h in range(2):
            for j in range(n):
                i, k = (2 * j, 2 * j + 1) if adjacent else (j, j + n)
                z = complex(x[t, h, i], x[t, h, k]) * \
                    np.exp(1j * pos[axes[j], t] * [1.0, 0.3, 0.01][j])
                assert abs(complex(y[t, h, i], y[t, h, k]) - z) < 1e-12
    assert np.array_equal(y[..., 2 * n:], x[..., 2 * n:])      # the rest is copied
    # q . k depends on the difference of the positions only
    q, k = x[:1], x[1:2]
    dot = [float((orope.rotate64(q, [a], table, None, adjacent) *
                  orope.rotate64(k, [b], table, None, adjacent)).sum()) for a, b in ((9, 4), (25, 20))]
    assert abs(dot[0] - dot[1]) < 1e-12
    # fp32: two products and a sum, each off by at most 2^-24 of itself
    z = orope.rotate(x.astype(np.float16), pos, table.astype(np.float32), axes, adjacent)
    ref = orope.rotate64(x.astype(np.float16), pos, table.astype(np.float32), axes, adjacent)
    assert z.dtype == np.float32 and np.abs(z - ref).max() <= 2 * np.abs(x).max() * 3 * 2.0 ** -24


def test_tables_and_sections():
    f = 10000.0 ** (-np.arange(64) / 64)
    t = real_ops.rope_table(f, 70000, magnitude=1.25, device="cpu")
    ref = orope.table64(f, 70000, 1.25)
    # rounded to fp32 once; fp64 angles and cosines are far finer
    assert t.dtype is F32 and np.abs(t.numpy() - ref).max() <= 1.25 * 2.0 ** -24 + 1e-10
    with pytest.raises(ValueError):
        real_ops.rope_table(f, 0, device="cpu")
    with pytest.raises(ValueError):
        real_ops.rope_table([[1.0]], 4, device="cpu")
    assert real_ops.rope_sections((2, 1, 3)) == (0, 0, 1, 2, 2, 2)
    assert real_ops.rope_sections((2, 1, 3), round_robin=True) == (0, 1, 2, 0, 2, 2)
    assert len(real_ops.rope_sections((16, 24, 24))) == 64


def test_entry_points_refuse_without_a_gpu(native_lib):
    L = native_lib
    p = 4096   # any aligned address: refused before it is used
    host = bytes([0, 1, 2, 3] * 16)

    def rotary(T=4, Hq=8, Hkv=2, D=128, q=p, k=p, ko=p, so=1024, sq=1024, sk=256, sko=256, pos=p,
               A=1, axes=None, table=p, rows=100, rot=128):
        return L.pkv_rotary_embedding(p, ko, q, k, so, sko, sq, sk, pos, A, axes, table, rows, rot,
                                      0, T, Hq, Hkv, D, None, None)

    def append(T=4, S=1, Hq=8, Hkv=2, D=128, bs=16, nb=8, mb=4, q=p, kc=p, qs=p, so=1024, sk=256,
               pos=None, A=1, axes=None, table=p, rows=100, rot=128):
        return L.pkv_rope_and_cache(p, q, p, p, so, 1024, sk, 256, qs, p, p, kc, p, pos, A, axes,
                                    table, rows, rot, 0, T, S, Hq, Hkv, D, bs, nb, mb, None, None)

    def append_q8(T=4, S=1, Hq=8, Hkv=2, D=128, bs=16, nb=8, mb=4, q=p, kc=p, ks=p, code=0,
                  stride=4, so=1024, sk=256, rows=100, rot=128, table=p, qs=p, pos=None, A=1,
                  axes=None):
        return L.pkv_rope_and_cache_q8(p, q, p, p, so, 1024, sk, 256, qs, p, p, kc, p, ks, p, code,
                                       pos, A, axes, table, rows, rot, 0, T, S, Hq, Hkv, D, bs, nb,
                                       mb, stride, None, None)

    assert rotary(T=0) == 0 and append(T=0) == 0 and append(S=0) == 0 and append_q8(T=0) == 0
    assert rotary(T=-1) == -1 and rotary(Hq=0) == -1 and rotary(Hkv=-1) == -1
    assert rotary(pos=None) == -1 and rotary(q=None) == -1 and rotary(ko=None) == -1
    assert rotary(q=p + 8) == -1 and rotary(pos=p + 2) == -1 and rotary(k=p + 2) == -1
    assert rotary(sko=128) == -1                # the outputs of two tokens overlap
    for call in (rotary, append, append_q8):
        assert call(D=64) == -2 and call(rot=24) == -2 and call(rot=144) == -2 and call(rot=0) == -1
        assert call(rows=0) == -1 and call(rows=2 ** 31) == -2 and call(A=0) == -1 and call(A=5) == -2
        assert call(A=2, axes=host) == -1           # an axis that is not there
        assert call(table=None) == -1 and call(table=p + 8) == -1
        assert call(so=1020) == -1 and call(sk=4) == -1 and call(so=896) == -1 and call(so=-1024) == -1
        assert call(Hq=2 ** 21) == -2
    for call in (append, append_q8):
        assert call(T=-1) == -1 and call(S=-1) == -1 and call(nb=0) == -1 and call(mb=0) == -1
        assert call(Hkv=0) == -1 and call(q=None) == -1 and call(kc=None) == -1 and call(qs=None) == -1
        assert call(kc=p + 8) == -1 and call(qs=p + 2) == -1
        assert call(nb=2 ** 31) == -2 and call(mb=2 ** 28) == -2
    assert append(bs=0) == -1 and append_q8(bs=0) == -1 and append_q8(bs=12) == -2
    assert append_q8(code=2) == -1 and append_q8(stride=1) == -1
    assert append_q8(ks=None) == -1 and append_q8(ks=p + 2) == -1


class Fake:
    """As much of a tensor on device 0 as the entry points look at."""

    def __init__(self, shape, dtype, device=0, stride=None, contiguous=True):
        self.shape, self.dtype, self.index, self.whole = torch.Size(shape), dtype, device, contiguous
        self.steps = stride or tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))
        self.device, self.is_cuda, self.ndim = "cuda:%d" % device, True, len(shape)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.whole

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.steps

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 4096


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *args: made.append((name, args)) or 0
    monkeypatch.setattr(real_ops, "lib", lambda: Recorder())
    monkeypatch.setattr(real_ops, "_get_device", lambda: 0)
    monkeypatch.setattr(real_ops, "_stream_handle", lambda stream: 0)
    return made


def arguments():
    T = 5
    qkv = lambda H: Fake((T, H, 128), F16, stride=(12 * 128, 128, 1))   # noqa: E731
    same = {"q_out": Fake((T, 8, 128), F16), "q": qkv(8), "table": Fake((99, 64, 2), F32)}
    cache = dict(same, k=qkv(2), v=qkv(2), query_start=Fake((3,), I32),
                 block_tables=Fake((2, 4), I32), context_lens=Fake((2,), I32))
    return {
        "rotary_embedding": dict(same, k_out=Fake((T, 2, 128), F16), k=qkv(2),
                                 positions=Fake((T,), I32)),
        "rope_and_cache": dict(cache, k_cache=Fake((9, 16, 2, 128), F16),
                               v_cache=Fake((9, 16, 2, 128), F16)),
        "rope_and_cache_q8": dict(cache, k_cache=Fake((9, 16, 2, 128), torch.int8),
                                  v_cache=Fake((9, 16, 2, 128), torch.int8),
                                  k_scale=Fake((9, 4), F32), v_scale=Fake((9, 4), F32)),
    }


NAMES = list(arguments())


@pytest.mark.parametrize("name", NAMES)
def test_wrappers_take_slices_and_refuse(calls, name):
    fn, good = getattr(real_ops, name), arguments()[name]
    T = 5
    fn(**good)
    fn(**good, dev_err=Fake((1,), I32), prepare=True)()
    assert [c[0] for c in calls] == ["pkv_" + name] * 2
    strides = calls[0][1][4:8]
    assert strides == ((1024, 256, 1536, 1536) if name == "rotary_embedding" else
                       (1024, 1536, 1536, 1536))
    fn(**dict(good, positions=Fake((3, T), I32)), axes=real_ops.rope_sections((16, 24, 24)))
    fn(**dict(good, positions=Fake((1, T), I32)), adjacent=True)
    fn(**dict(good, positions=Fake((3, T), I32)), axes=[2] * 64)
    del calls[:]
    rows = lambda H=8, **a: Fake((T, H, 128), F16, **a)      # noqa: E731
    bad = [dict(q=rows(stride=(1536, 128, 2))), dict(q=rows(stride=(1536, 256, 1))),
           dict(q=rows(stride=(1028, 128, 1))), dict(q=rows(7)), dict(q=rows(device=1)),
           dict(q=Fake((T, 8, 64), F16)), dict(q=Fake((T, 8, 128), F32)), dict(q=None),
           dict(q=torch.zeros(T, 8, 128, dtype=F16)), dict(q=Fake((T, 1024), F16)),
           dict(q_out=rows(stride=(896, 128, 1))), dict(q_out=Fake((T + 1, 8, 128), F16)),
           dict(k=rows(3)), dict(k=Fake((T - 1, 2, 128), F16)),
           dict(table=Fake((99, 64), F32)), dict(table=Fake((99, 64, 3), F32)),
           dict(table=Fake((99, 64, 2), F16)), dict(table=Fake((99, 64, 2), F32, contiguous=False)),
           dict(table=None), dict(positions=Fake((T + 1,), I32)), dict(positions=Fake((T,), torch.int64)),
           dict(positions=Fake((5, T), I32), axes=(0,) * 64), dict(positions=Fake((3, T), I32)),
           dict(positions=Fake((2, T), I32), axes=real_ops.rope_sections((16, 24, 24))),
           dict(positions=Fake((3, T), I32), axes=real_ops.rope_sections((16, 24, 23))),
           dict(positions=Fake((3, T), I32), axes=(-1,) * 64),
           dict(positions=Fake((T,), I32, contiguous=False)), dict(positions=torch.zeros(T, dtype=I32)),
           dict(dev_err=Fake((1,), torch.int64)), dict(dev_err=torch.zeros(1, dtype=I32))]
    if name == "rotary_embedding":
        bad += [dict(positions=None), dict(k=None), dict(k_out=None), dict(k_out=rows(3)),
                dict(k_out=rows(2, stride=(128, 128, 1)))]
    else:
        bad += [dict(v=rows(3)), dict(query_start=Fake((4,), I32)), dict(context_lens=Fake((3,), I32)),
                dict(block_tables=Fake((2,), I32)), dict(block_tables=Fake((2, 4), torch.int64)),
                dict(k_cache=Fake((9, 16, 3, 128), good["k_cache"].dtype)),
                dict(v_cache=Fake((8, 16, 2, 128), good["k_cache"].dtype)),
                dict(k_cache=Fake((9, 16, 2, 128), F32)),
                dict(k_cache=Fake((9, 16, 2, 128), good["k_cache"].dtype, contiguous=False))]
    if name == "rope_and_cache_q8":
        bad += [dict(k_scale=Fake((9, 1), F32)), dict(v_scale=Fake((9, 8), F32)),
                dict(k_scale=Fake((8, 4), F32))]
    for change in bad:
        with pytest.raises((TypeError, ValueError)):
            fn(**{**good, **change})
    assert calls == []
    if name == "rotary_embedding":
        fn(**dict(good, k=None, k_out=None))
        fn(**dict(good, q_out=good["q"], k_out=good["k"]))        # in place
        assert len(calls) == 2
