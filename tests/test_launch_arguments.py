"""The workspace and error word that a caller brings to the prompt and 8-bit entry points: a kernel
writes them, so what is not memory of the current device, or is not laid out as it is taken to be,
is refused before a launch.  Stand-ins for CUDA tensors and a library that only records: no GPU.
"""
import pytest
import torch

from paged_kv_cache_138_gb300 import ops as real_ops

F16, I32, F32 = torch.float16, torch.int32, torch.float32


class Fake:
    """As much of a contiguous tensor on device 0 as the entry points look at."""

    def __init__(self, shape, dtype, device=0, contiguous=True):
        self.shape, self.dtype, self.index, self.whole = torch.Size(shape), dtype, device, contiguous
        self.device, self.is_cuda = "cuda:%d" % device, True

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.whole

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def data_ptr(self):
        return 4096


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def ops(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(real_ops, "lib", lambda: rec)
    monkeypatch.setattr(real_ops, "_get_device", lambda: 0)
    monkeypatch.setattr(real_ops, "_stream_handle", lambda stream: 0)
    monkeypatch.setattr(real_ops, "prefill_workspace_bytes", lambda *a: 0)
    monkeypatch.setattr(real_ops, "workspace_bytes", lambda *a: 0)
    return real_ops, rec


def entry_points(ops):
    q, k = Fake((2, 8, 128), F16), Fake((2, 2, 128), F16)
    kc, tab, lens, qs = Fake((4, 16, 2, 128), F16), Fake((1, 4), I32), Fake((1,), I32), Fake((2,), I32)
    q8 = (Fake((4, 16, 2, 128), torch.int8),) * 2 + (Fake((4, 4), F32),) * 2
    one = Fake((1, 8, 128), F16)
    return {
        "paged_attention_prefill": lambda **a: ops.paged_attention_prefill(q, q, kc, kc, tab, lens,
                                                                           qs, 1.0, **a),
        "prompt_attention": lambda **a: ops.prompt_attention(q, q, k, k, qs, 1.0, **a),
        "reshape_and_cache_q8": lambda **a: ops.reshape_and_cache_q8(k, k, qs, tab, lens, *q8, **a),
        "paged_attention_decode_q8": lambda **a: ops.paged_attention_decode_q8(one, one, *q8, tab,
                                                                               lens, 1.0, **a),
    }


NAMES = ["paged_attention_prefill", "prompt_attention", "reshape_and_cache_q8",
         "paged_attention_decode_q8"]


@pytest.mark.parametrize("prepare", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_error_word(ops, name, prepare):
    ops, rec = ops
    call = entry_points(ops)[name]
    bad = [(torch.zeros(1, dtype=I32), TypeError),              # of the host
           (torch.zeros(1, dtype=I32, device="meta"), TypeError),
           (Fake((1,), torch.int64), TypeError),
           (Fake((1,), torch.uint8), TypeError),
           (Fake((1,), I32, device=1), (TypeError, ValueError)),
           (Fake((4,), I32, contiguous=False), (TypeError, ValueError)),
           (Fake((0,), I32), (TypeError, ValueError)),
           (4096, TypeError)]
    for err, kind in bad:
        with pytest.raises(kind):
            call(dev_err=err, prepare=prepare)
    assert rec.calls == []
    call(dev_err=Fake((1,), I32))
    call()
    assert rec.calls == ["pkv_" + name] * 2


@pytest.mark.parametrize("prepare", [False, True])
@pytest.mark.parametrize("name", [NAMES[0], NAMES[3]])
def test_workspace(ops, name, prepare):
    ops, rec = ops
    call = entry_points(ops)[name]
    bad = [(torch.zeros(64, dtype=torch.uint8), TypeError),
           (torch.zeros(64, dtype=torch.uint8, device="meta"), TypeError),
           (Fake((64,), torch.uint8, device=1), (TypeError, ValueError)),
           (Fake((64,), torch.uint8, contiguous=False), (TypeError, ValueError)),
           (4096, TypeError)]
    for ws, kind in bad:
        with pytest.raises(kind):
            call(workspace=ws, prepare=prepare)
    assert rec.calls == []
    call(workspace=Fake((64,), torch.uint8))
    call(workspace=Fake((64,), F32))
    assert rec.calls == ["pkv_" + name] * 2
