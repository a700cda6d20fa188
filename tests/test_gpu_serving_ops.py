"""The prompt and 8-bit-cache operators in one run, as a server uses them: prompts
attended and written, then decode steps that write and attend, with block tables from
the BlockManager; and a prompt taken in chunks over the fp16 cache."""
import numpy as np
import pytest
import torch

import test_gpu_prompt as tp
import test_gpu_q8 as tq
from oracle import prompt as op
from oracle import q8 as oq
from paged_kv_cache_138_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
D = 128
SCALE = 1.0 / np.sqrt(D)


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_prompts_then_decode_on_the_8bit_cache(ops, code):
    from paged_kv_cache_138_gb300.block_manager import BlockManager
    rng = np.random.default_rng(31)
    Hq, Hkv, bs, nb, mb = 8, 2, 16, 160, 48
    bm = BlockManager(nb, bs, enable_prefix_cache=False)
    prompts = [150, 33, 1, 300]
    for s, n in enumerate(prompts):
        bm.allocate(s, rng.integers(0, 32000, size=n).tolist())
    tables, lens = bm.block_tables([0, 1, 2, 3], max_blocks=mb)
    kc, vc, ks, vs = ops.q8_cache(nb, Hkv, bs, tq.DTYPE[code])
    err = ops.new_error_word()
    qs = tp.starts(prompts)
    T = int(qs[-1])
    q = wl.host_normal_fp16(rng, (T, Hq, D))
    k, v = (wl.host_normal_fp16(rng, (T, Hkv, D)) for _ in "kv")
    out = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda")
    qd, kd, vd, qsd = dev(q), dev(k), dev(v), dev(qs)
    ops.prompt_attention(out, qd, kd, vd, qsd, SCALE, dev_err=err)
    ops.reshape_and_cache_q8(kd, vd, qsd, dev(tables), dev(lens), kc, vc, ks, vs, dev_err=err)
    assert ops.read_error_word(err) == 0
    got = out.cpu().numpy()
    for s in range(4):
        a, b = qs[s], qs[s + 1]
        tp.check(got[a:b], q[a:b], k[a:b], v[a:b], 0)
    codes = [np.zeros((nb, bs, Hkv, D)) for _ in "kv"]
    scales = [np.zeros((nb, 4), np.float32) for _ in "kv"]
    for x, c, sc in zip((k, v), codes, scales):
        oq.write(x, qs, tables, lens, c, sc, bs, code)
    one = dev(tp.starts([1] * 4))
    o1 = torch.empty((4, Hq, D), dtype=torch.float16, device="cuda")
    for step in range(20):
        for s in range(4):
            bm.append_slot(s, int(rng.integers(0, 32000)))
        tables, lens = bm.block_tables([0, 1, 2, 3], max_blocks=mb)
        td, ld = dev(tables), dev(lens)
        x = [wl.host_normal_fp16(rng, (4, Hkv, D)) for _ in "kv"]
        q1 = wl.host_normal_fp16(rng, (4, Hq, D))
        ops.reshape_and_cache_q8(dev(x[0]), dev(x[1]), one, td, ld, kc, vc, ks, vs, dev_err=err)
        ops.paged_attention_decode_q8(o1, dev(q1), kc, vc, ks, vs, td, ld, SCALE, dev_err=err)
        for i in range(2):
            oq.write(x[i], tp.starts([1] * 4), tables, lens, codes[i], scales[i], bs, code)
        tq.check_decode(o1.cpu().numpy().astype(np.float64), q1, codes, scales, tables, lens, bs)
    assert ops.read_error_word(err) == 0
    assert np.array_equal(tq.codes_of(kc, code), codes[0])


def test_prompt_in_chunks_over_the_fp16_cache(ops):
    """A prompt written and attended chunk by chunk gives the rows of the whole prompt's
    attention, and decode attention goes on from there."""
    rng = np.random.default_rng(32)
    Hq, Hkv, bs, n = 16, 4, 16, 700
    nb = 60
    table = rng.permutation(nb).astype(np.int32)[None, :wl.blocks_for(n + 1, bs)]
    kc = torch.full((nb, bs, Hkv, D), float("nan"), dtype=torch.float16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    q = wl.host_normal_fp16(rng, (n + 1, Hq, D))
    k, v = (wl.host_normal_fp16(rng, (n + 1, Hkv, D)) for _ in "kv")
    qd, kd, vd, td = dev(q), dev(k), dev(v), dev(table)
    err = ops.new_error_word()
    rows = []
    for a, b in ((0, 1), (1, 17), (17, 300), (300, 556), (556, 700)):
        pos = np.arange(a, b)
        slots = table[0][pos // bs].astype(np.int64) * bs + pos % bs
        ops.reshape_and_cache(kd[a:b], vd[a:b], dev(slots), kc, vc, dev_err=err)
        out = torch.empty_like(qd[a:b])
        ops.paged_attention_prefill(out, qd[a:b], kc, vc, td, dev(np.array([b], np.int32)),
                                    dev(np.array([0, b - a], np.int32)), SCALE, dev_err=err)
        rows.append(out)
    got = torch.cat(rows).cpu().numpy()
    tp.check(got, q[:n], k[:n], v[:n], 0)
    whole = torch.empty_like(qd[:n])
    ops.prompt_attention(whole, qd[:n], kd[:n], vd[:n], dev(np.array([0, n], np.int32)), SCALE,
                         dev_err=err)
    tp.check(whole.cpu().numpy(), q[:n], k[:n], v[:n], 0)
    out = torch.empty_like(qd[n:])
    ops.paged_attention_decode_fused(out, qd[n:], kd[n:], vd[n:], kc, vc, td,
                                     dev(np.array([n + 1], np.int32)), SCALE, dev_err=err)
    tp.check(out.cpu().numpy(), q[n:], k, v, n)
    assert ops.read_error_word(err) == 0
    assert op.gather(kc.cpu().numpy(), table[0], n + 1).shape == k.shape


def test_two_streams_at_once(ops):
    """Prompts on one stream and decode steps on another, at the same time, on caches and
    workspaces of their own: the results of each alone."""
    q, kc, vc, tables, lens = tp.paged_case(33, [6, 300], [3000, 100], 8, 2, 16)
    args = [dev(a) for a in (q, kc, vc, tables, lens, tp.starts([6, 300]))]
    dq, codes, scales, dtab, dlens = tq.decode_case(34, [2500, 40, 700], 8, 2, 16, "int8")
    dargs = [dev(dq)] + [tq.codes_to_dev(c, "int8") for c in codes] + [dev(s) for s in scales] + \
        [dev(dtab), dev(dlens)]
    outs = [torch.zeros_like(args[0]) for _ in range(2)]
    douts = [torch.zeros_like(dargs[0]) for _ in range(2)]
    ops.paged_attention_prefill(outs[0], *args, SCALE)
    ops.paged_attention_decode_q8(douts[0], *dargs, SCALE)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    n = ops.prefill_workspace_bytes(q.shape[0], 2, 8, 2, tables.shape[1])
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    dws = ops.alloc_workspace(3, 8, dtab.shape[1])
    torch.cuda.synchronize()
    for _ in range(10):
        ops.paged_attention_prefill(outs[1], *args, SCALE, workspace=ws, stream=streams[0])
        ops.paged_attention_decode_q8(douts[1], *dargs, SCALE, workspace=dws, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(douts[0], douts[1])


@pytest.mark.parametrize("raw", [False, True])
def test_own_workspace_belongs_to_the_launch_stream(ops, raw):
    """A workspace made by the call is of the stream it launches on: given back, it must not
    go to work of the current stream while the launch still runs."""
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    z = lambda *s, dtype=torch.float16: torch.zeros(s, dtype=dtype, device="cuda")
    kc, tab = z(2048, 16, 2, 128), torch.arange(2048, dtype=torch.int32, device="cuda")[None]
    lens = torch.full((1,), 32768, dtype=torch.int32, device="cuda")
    q, qs = z(8, 8, 128), torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    k8 = ops.q8_cache(2048, 2)
    calls = [(ops.prefill_workspace_bytes(8, 1, 8, 2, 2048), lambda: ops.paged_attention_prefill(
                  torch.empty_like(q), q, kc, kc, tab, lens, qs, 1.0, stream=stream, prepare=True)),
             (ops.workspace_bytes(1, 8, 2048), lambda: ops.paged_attention_decode_q8(
                  z(1, 8, 128), z(1, 8, 128), *k8, tab, lens, 1.0, stream=stream, prepare=True))]
    for need, prepare in calls:
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


def test_tensors_of_another_device_are_refused(ops, monkeypatch):
    """The kernels run on the current device; a tensor elsewhere is refused before a launch."""
    z = lambda *s, dtype=torch.float16: torch.zeros(s, dtype=dtype, device="cuda")
    q, kc = torch.full((2, 8, 128), 3.0, dtype=torch.float16, device="cuda"), z(4, 16, 2, 128)
    tab, lens = z(1, 4, dtype=torch.int32), torch.full((1,), 2, dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    k, k8, out = z(2, 2, 128), ops.q8_cache(4, 2), z(2, 8, 128)
    calls = [lambda: ops.prompt_attention(out, q, k, k, qs, 1.0),
             lambda: ops.paged_attention_prefill(out, q, kc, kc, tab, lens, qs, 1.0),
             lambda: ops.reshape_and_cache_q8(k, k, qs, tab, lens, *k8),
             lambda: ops.paged_attention_decode_q8(out[:1], q[:1], *k8, tab, lens, 1.0)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(ops, "_get_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
