"""A workspace that an fp16 decode call makes is of the stream it launches on: given back when the
call returns, it must not go to work of the current stream while the launch still runs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def z(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["decode", "fused", "grouped", "grouped_fused"])
def test_own_workspace_belongs_to_the_launch_stream(ops, name, raw):
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    kc, tab = z(2048, 16, 2, 128), torch.arange(2048, dtype=torch.int32, device="cuda")[None]
    lens = torch.full((1,), 32768, dtype=torch.int32, device="cuda")
    q, new = z(1, 8, 128), z(1, 2, 128)
    groups = (torch.tensor([0, 1], dtype=torch.int32, device="cuda"), z(1, dtype=torch.int32),
              z(1, dtype=torch.int32), 0, 32768)
    last = dict(stream=stream, prepare=True)
    prepare = {
        "decode": lambda: ops.paged_attention_decode(z(1, 8, 128), q, kc, kc, tab, lens, 1.0, **last),
        "fused": lambda: ops.paged_attention_decode_fused(z(1, 8, 128), q, new, new, kc, kc, tab,
                                                          lens, 1.0, **last),
        "grouped": lambda: ops.paged_attention_decode_grouped(z(1, 8, 128), q, kc, kc, tab, lens,
                                                              *groups, 1.0, **last),
        "grouped_fused": lambda: ops.paged_attention_decode_grouped_fused(
            z(1, 8, 128), q, new, new, kc, kc, tab, lens, *groups, 1.0, **last),
    }[name]
    need = ops.grouped_workspace_bytes(1, 8, 2048, 0) if "grouped" in name else \
        ops.workspace_bytes(1, 8, 2048)
    assert need > 0
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    launch = prepare()
    used = [t.data_ptr() for t in launch._keep if isinstance(t, torch.Tensor) and
            t.dtype is torch.uint8 and t.numel() == need]
    assert len(used) == 1
    del launch
    mine = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert used[0] not in [t.data_ptr() for t in mine]
    with torch.cuda.stream(torch.cuda.ExternalStream(side.cuda_stream)):
        theirs = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert used[0] in [t.data_ptr() for t in theirs]
