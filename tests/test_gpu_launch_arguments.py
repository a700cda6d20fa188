"""Workspaces and error words of the prompt and 8-bit entry points, with CUDA tensors: good ones
are taken, others refused with the launch not made (out stays as it was)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def z(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def test_workspace_and_error_word(ops, monkeypatch):
    q, k, out = z(2, 8, 128), z(2, 2, 128), torch.full((2, 8, 128), 3.0, dtype=torch.float16,
                                                       device="cuda")
    kc, tab = z(4, 16, 2, 128), z(1, 2048, dtype=torch.int32)
    lens = torch.full((1,), 2, dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    k8 = ops.q8_cache(4, 2)
    calls = [lambda **a: ops.prompt_attention(out, q, k, k, qs, 1.0, **a),
             lambda **a: ops.reshape_and_cache_q8(k, k, qs, tab, lens, *k8, **a)]
    split = [(ops.prefill_workspace_bytes(2, 1, 8, 2, 2048),
              lambda **a: ops.paged_attention_prefill(out, q, kc, kc, tab, lens, qs, 1.0, **a)),
             (ops.workspace_bytes(1, 8, 2048),
              lambda **a: ops.paged_attention_decode_q8(out[:1], q[:1], *k8, tab, lens, 1.0, **a))]
    for call in calls + [c for _, c in split]:
        for err in (z(1, dtype=torch.int64), z(8, dtype=torch.int32)[::2], z(0, dtype=torch.int32),
                    torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32).pin_memory()):
            with pytest.raises((TypeError, ValueError)):
                call(dev_err=err)
    for need, call in split:
        assert need > 0
        for ws in (torch.zeros(need, dtype=torch.uint8), z(need, 2, dtype=torch.uint8)[:, 0],
                   z(need // 4, 4, dtype=torch.uint8).t()):
            with pytest.raises((TypeError, ValueError)):
                call(workspace=ws)
    assert bool((out == 3).all()) and not any(bool(t.view(torch.uint8).any()) for t in k8)
    with monkeypatch.context() as m:
        m.setattr(ops, "_get_device", lambda: 1)
        with pytest.raises(ValueError, match="current CUDA device"):
            ops._check_side(None, z(1, dtype=torch.int32))
        with pytest.raises(ValueError, match="current CUDA device"):
            ops._check_side(z(16, dtype=torch.uint8), None)
    err = ops.new_error_word()
    for need, call in split:
        call(dev_err=err, workspace=z(need // 4, dtype=torch.float32))
    for call in calls:
        call(dev_err=err)
    assert ops.read_error_word(err) == 0 and not bool((out == 3).any())
