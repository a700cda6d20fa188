"""The prompt and 8-bit kernels' bounded waits on a barrier nothing arrives on: they run out after
their limit, say so and return; the GPU keeps working."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def test_waits_give_up_and_report(ops, native_lib):
    err, out = ops.new_error_word(), torch.full((5,), 7, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for bad in (0, -1, 2 ** 31 + 1):
        assert native_lib.pkv_selftest_warp_waits(err.data_ptr(), out.data_ptr(), bad, stream) == -1
    assert native_lib.pkv_selftest_warp_waits(None, out.data_ptr(), 10 ** 8, stream) == -1
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert native_lib.pkv_selftest_warp_waits(err.data_ptr(), out.data_ptr(), 10 ** 8, stream) == 0
    assert ops.read_error_word(err) == 4          # PKV_DEV_WAIT_TIMEOUT
    # two waits of 10^8 cycles, at no more than 2.07 GHz
    assert 2 * 10 ** 8 / 2.07e9 <= time.perf_counter() - t0 < 10
    assert out.tolist() == [1, 1, 0, 0, 1]
    q = torch.randn((300, 2, 128), device="cuda").half()
    qs = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    o, err2 = torch.full_like(q, float("nan")), ops.new_error_word()
    ops.prompt_attention(o, q, q, q, qs, 0.1, dev_err=err2)
    assert ops.read_error_word(err2) == 0 and bool(torch.isfinite(o).all())
