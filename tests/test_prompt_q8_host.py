"""8-bit prompt attention on the host: its oracle against the fp16 one's, the C entry point's
refusals (no CUDA call is made) and the wrapper's (stand-ins for CUDA tensors)."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from oracle import q8 as oq
from paged_kv_cache_138_gb300 import ops as real_ops
from test_rope_host import Fake, calls  # noqa: F401

F16, F32, I32 = torch.float16, torch.float32, torch.int32


def test_oracle_is_attention_over_the_values():
    rng = np.random.default_rng(0)
    q = rng.standard_normal((5, 4, 8))
    kc, vc = (np.round(rng.uniform(-127, 127, (9, 2, 8))) for _ in "kv")
    ks, vs = (rng.uniform(0.01, 0.02, (9, 2)) for _ in "kv")
    got = oq.chunk(q, kc, vc, ks, vs, 4, 0.3)
    ref = op.attend(q, kc * ks[:, :, None], vc * vs[:, :, None], 4, 0.3)
    assert np.abs(got[0] - ref[0]).max() < 1e-12 and np.abs(got[1] - ref[1]).max() < 1e-12
    assert np.abs(got[3] - ref[3]).max() < 1e-12 and (got[2] <= ref[2] * vs.max() + 1e-15).all()


def test_entry_point_refuses_without_a_gpu(native_lib):
    p = 4096   # any aligned address: refused before it is used

    def run(T=4, S=1, Hq=8, Hkv=2, D=128, bs=16, nb=8, mb=4, stride=4, code=0, q=p, kc=p, ks=p, t=p,
            n=p, qs=p, ws=None, b=0):
        return native_lib.pkv_paged_attention_prefill_q8(
            p, q, kc, p, ks, p, code, t, n, qs, T, S, Hq, Hkv, D, bs, nb, mb, stride, 0.1, ws, b,
            None, None)

    assert run(T=0) == 0 and run(S=0) == 0
    assert run(T=-1) == -1 and run(S=-1) == -1 and run(Hq=0) == -1 and run(nb=0) == -1
    assert run(mb=0) == -1 and run(stride=1) == -1 and run(code=2) == -1
    for name in ("q", "kc", "ks", "t", "n", "qs"):
        assert run(**{name: None}) == -1
    assert run(q=p + 8) == -1 and run(kc=p + 8) == -1 and run(ks=p + 2) == -1
    assert run(D=64) == -2 and run(Hq=6, Hkv=4) == -2 and run(Hq=32, Hkv=2) == -2
    for bs in (0, 4, 12, 128):
        assert run(bs=bs) == -2
    assert run(nb=2 ** 31) == -2 and run(mb=2 ** 22) == -2
    need = native_lib.pkv_paged_attention_prefill_q8_workspace_bytes(8, 1, 32, 8, 2048, 16)
    assert need > 0
    few = dict(T=8, Hq=32, Hkv=8, mb=2048, stride=8)
    assert run(**few) == -1 and run(**few, ws=p, b=need - 1) == -1 and run(**few, ws=p + 8, b=need) == -1


def test_wrapper_refuses(calls, monkeypatch):   # noqa: F811
    monkeypatch.setattr(real_ops, "prefill_q8_workspace_bytes", lambda *a: 0)
    i8 = torch.int8
    good = dict(out=Fake((5, 8, 128), F16), q=Fake((5, 8, 128), F16), k_cache=Fake((9, 16, 2, 128), i8),
                v_cache=Fake((9, 16, 2, 128), i8), k_scale=Fake((9, 4), F32),
                v_scale=Fake((9, 4), F32), block_tables=Fake((2, 4), I32),
                context_lens=Fake((2,), I32), query_start=Fake((3,), I32), scale=0.1)
    fn = real_ops.paged_attention_prefill_q8
    fn(**good)
    fn(**good, prepare=True, dev_err=Fake((1,), I32))()
    assert [c[0] for c in calls] == ["pkv_paged_attention_prefill_q8"] * 2
    del calls[:]
    for change in (dict(q=Fake((5, 8, 128), F32)), dict(q=Fake((5, 8, 128), F16, contiguous=False)),
                   dict(q=Fake((5, 8, 128), F16, device=1)), dict(q=Fake((4, 8, 128), F16)), dict(q=None),
                   dict(out=Fake((5, 8, 64), F16)), dict(out=torch.zeros(5, 8, 128, dtype=F16)),
                   dict(k_cache=Fake((9, 16, 2, 128), F16)), dict(v_cache=Fake((8, 16, 2, 128), i8)),
                   dict(k_scale=Fake((9, 1), F32)), dict(k_scale=Fake((9, 4), F16)),
                   dict(block_tables=Fake((2, 4), torch.int64)), dict(block_tables=Fake((3, 4), I32)),
                   dict(context_lens=Fake((3,), I32)), dict(query_start=Fake((2,), I32)),
                   dict(workspace=torch.zeros(8, dtype=torch.uint8)), dict(dev_err=Fake((1,), F32))):
        with pytest.raises((TypeError, ValueError)):
            fn(**{**good, **change})
    assert calls == []


@pytest.mark.parametrize("T,S,Hq,Hkv", [(1, 1, 8, 8), (26, 4, 32, 8), (512, 16, 32, 8), (800, 8, 32, 32),
                                        (2048, 4, 32, 8), (256, 256, 32, 8), (40, 1, 64, 8)])
@pytest.mark.parametrize("width", [1, 8, 9, 64, 2048, 1 << 21])
def test_workspace_is_whole_splits(native_lib, T, S, Hq, Hkv, width):
    """Partials of 130 floats a row and split, no more splits than the table has tiles of 128
    tokens, none where it has one."""
    need = native_lib.pkv_paged_attention_prefill_q8_workspace_bytes(T, S, Hq, Hkv, width, 16)
    splits, rest = divmod(need, T * Hq * 130 * 4)
    tiles = -(-width * 16 // 128)
    assert rest == 0 and splits != 1 and splits <= tiles
    if tiles == 1:
        assert need == 0


@pytest.mark.parametrize("T,S,Hq,Hkv", [(1, 1, 8, 8), (26, 4, 32, 8), (40, 1, 64, 8), (100, 2, 8, 8)])
@pytest.mark.parametrize("width", [2048, 16384])
def test_few_rows_over_long_contexts_are_split(native_lib, T, S, Hq, Hkv, width):
    """The key axis is cut where the rows alone leave SMs idle, and a workspace that is short by a
    byte, or none, is refused."""
    need = native_lib.pkv_paged_attention_prefill_q8_workspace_bytes(T, S, Hq, Hkv, width, 16)
    splits = need // (T * Hq * 130 * 4)
    assert splits > 1
    p = 4096

    def run(ws, b):
        return native_lib.pkv_paged_attention_prefill_q8(
            p, p, p, p, p, p, 0, p, p, p, T, S, Hq, Hkv, 128, 16, 64, width, -(-Hkv // 4) * 4, 0.1,
            ws, b, None, None)
    assert run(p, need - 1) == -1 and run(None, need) == -1 and run(p + 8, need) == -1
