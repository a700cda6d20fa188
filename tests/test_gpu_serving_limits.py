"""Prompt attention and the 8-bit cache at sizes where an index can overflow.

* Pools of more than 2^32 bytes (fp16: of more than 2^32 elements), the blocks in use spread
  over all of it, the last one among them: the same bits as in a small pool.
* 65,535 sequences in one decode launch (65,536 are refused): the same bits as in
  launches of 8,192.
* Contexts of 2^20 + 7 tokens with three equal dominant keys, in the first, a middle and
  the last split: against fp64, with the tolerances derived in test_gpu_prompt.py
  and test_gpu_q8.py.
* Metadata that is out of range, with no error word to report it in.
"""
import numpy as np
import pytest
import torch

import test_gpu_prompt as tp
import test_gpu_q8 as tq
from oracle import prompt as op
from paged_kv_cache_138_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
D = 128
SCALE = 1.0 / np.sqrt(D)
LONG = 2 ** 20 + 7


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def spread_tables(rng, small, blocks):
    """The table `small` with its ids moved to `blocks` blocks, the last one among them."""
    ids = np.unique(small[small >= 0])
    to = np.sort(rng.choice(blocks - 1, len(ids), replace=False)).astype(np.int32)
    to[-1] = blocks - 1
    at = dict(zip(ids.tolist(), to.tolist()))
    return np.vectorize(lambda b: at.get(b, -9), otypes=[np.int32])(small), ids, to


@pytest.mark.parametrize("bs", [16, 64])
def test_prefill_in_a_pool_of_2_32_elements(ops, bs):
    new, cached = [9, 130, 1], [400, 0, 2000]
    q, kc, vc, tables, lens = tp.paged_case(bs, new, cached, 8, 2, bs, poison=False)
    err = ops.new_error_word()
    rest = [dev(lens), dev(tp.starts(new)), SCALE]
    want = torch.zeros(q.shape, dtype=torch.float16, device="cuda")
    ops.paged_attention_prefill(want, dev(q), dev(kc), dev(vc), dev(tables), *rest, dev_err=err)
    blocks = 2 ** 32 // (bs * 2 * D) + 5
    far, ids, to = spread_tables(np.random.default_rng(1), tables, blocks)
    pools = [torch.empty((blocks, bs, 2, D), dtype=torch.float16, device="cuda") for _ in "kv"]
    for pool, c in zip(pools, (kc, vc)):
        pool[dev(to.astype(np.int64))] = dev(c[ids])
    got = torch.zeros_like(want)
    ops.paged_attention_prefill(got, dev(q), *pools, dev(far), *rest, dev_err=err)
    assert ops.read_error_word(err) == 0
    assert torch.equal(got, want)
    tp.check_paged(got.cpu().numpy(), q, kc, vc, tables, lens, new)


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_8bit_cache_in_a_pool_of_2_32_bytes(ops, dtype):
    rng = np.random.default_rng(2)
    new, bs = [300, 1, 17], 16
    lens = new
    nb, tables = tq.batch(rng, lens, bs)
    k, v = (dev(wl.host_normal_fp16(rng, (sum(new), 2, D))) for _ in "kv")
    q = dev(wl.host_normal_fp16(rng, (3, 8, D)))
    qs, n = dev(tp.starts(new)), dev(np.asarray(lens, np.int32))
    blocks = 2 ** 32 // (bs * 2 * D) + 5
    far, ids, to = spread_tables(rng, tables, blocks)
    err, outs, rows = ops.new_error_word(), [], []
    for t, count, used in ((tables, nb, ids), (far, blocks, to)):
        stride = 4
        cache = [torch.empty((count, bs, 2, D), dtype=torch.uint8, device="cuda").view(dtype)
                 for _ in "kv"]
        scales = [torch.zeros((count, stride), dtype=torch.float32, device="cuda") for _ in "kv"]
        at = dev(np.asarray(used, np.int64))
        for c in cache:
            c.view(torch.uint8)[at] = 0
        ops.reshape_and_cache_q8(k, v, qs, dev(t), n, *cache, *scales, dev_err=err)
        out = torch.zeros_like(q)
        ops.paged_attention_decode_q8(out, q, *cache, *scales, dev(t), n, SCALE, dev_err=err)
        outs.append(out)
        rows.append([c.view(torch.uint8)[at] for c in cache] + [s[at] for s in scales])
        del cache, scales
    assert ops.read_error_word(err) == 0
    assert all(torch.equal(a, b) for a, b in zip(*rows))
    assert torch.equal(*outs) and bool(outs[0].abs().sum() > 0)


def test_largest_decode_batch(ops):
    S = 65535
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 32, S, endpoint=True).astype(np.int32)
    tables = rng.integers(0, 5000, (S + 1, 2)).astype(np.int32)
    kc, vc, ks, vs = ops.q8_cache(5000, 1)
    for c in (kc, vc):
        c.view(torch.uint8).random_(0, 255)
    for s in (ks, vs):
        s.uniform_(0.01, 0.03)
    q = dev(wl.host_normal_fp16(rng, (S + 1, 8, D)))
    t, n = dev(tables), dev(np.append(lens, np.int32(1)))
    err = ops.new_error_word()
    got, want = torch.zeros_like(q), torch.zeros_like(q)
    ops.paged_attention_decode_q8(got[:S], q[:S], kc, vc, ks, vs, t[:S], n[:S], SCALE, dev_err=err)
    for a in range(0, S, 8192):
        b = min(S, a + 8192)
        ops.paged_attention_decode_q8(want[a:b], q[a:b], kc, vc, ks, vs, t[a:b], n[a:b], SCALE,
                                      dev_err=err)
    assert ops.read_error_word(err) == 0
    assert torch.equal(got, want)
    from paged_kv_cache_138_gb300._lib import PagedKVError
    with pytest.raises(PagedKVError):
        ops.paged_attention_decode_q8(got, q, kc, vc, ks, vs, t, n, SCALE)


def test_8bit_decode_of_a_million_tokens(ops):
    q, codes, scales, tables, lens = tq.decode_case(5, [LONG], 2, 1, 16, "int8")
    qq = q[0, 0].astype(np.float64)
    key = np.rint(qq / np.abs(qq).max() * 127).astype(np.int64)
    for pos in (3, LONG // 2, LONG - 1):
        b, r = tables[0, pos // 16], pos % 16
        codes[0][b, r, 0] = key
        scales[0][b] = 0.5
    got, err = tq.run_decode(ops, q, codes, scales, tables, lens, "int8", 16)
    assert err == 0
    tq.check_decode(got, q, codes, scales, tables, lens, 16)


def test_prefill_behind_a_million_tokens(ops):
    new, cached = [3], [LONG - 3]
    q, kc, vc, tables, lens = tp.paged_case(6, new, cached, 2, 1, 16)
    for pos in (3, LONG // 2, LONG - 1):
        kc[tables[0, pos // 16], pos % 16, 0] = q[2, 0] * np.float16(2)
    got, err = tp.run_paged(ops, q, kc, vc, tables, lens, tp.starts(new))
    assert err == 0
    tp.check_paged(got, q, kc, vc, tables, lens, new)


def test_bad_metadata_without_an_error_word(ops):
    new, cached = [20, 33, 5], [0, 50, 7]
    q, kc, vc, tables, lens = tp.paged_case(7, new, cached, 8, 2, 16)
    bad_t, bad_n = tables.copy(), lens.copy()
    bad_t[0, 1], bad_n[1] = 10 ** 6, -3
    d = [dev(a) for a in (q, kc, vc, bad_t, bad_n, tp.starts(new))]
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    ops.paged_attention_prefill(out, *d, SCALE)
    got = out.cpu().numpy()
    assert (got[20:53] == 7).all()
    tp.check(got[53:58], q[53:58], op.gather(kc, tables[2], 12), op.gather(vc, tables[2], 12), 7)
    cache = ops.q8_cache(kc.shape[0], 2)
    k = dev(wl.host_normal_fp16(np.random.default_rng(8), (58, 2, D)))
    k[0, 0, 0] = float("inf")
    ops.reshape_and_cache_q8(k, k, d[5], d[3], d[4], *cache)
    one = torch.full((3, 8, D), 7.0, dtype=torch.float16, device="cuda")
    ops.paged_attention_decode_q8(one, d[0][:3].contiguous(), *cache, d[3], d[4], SCALE)
    assert bool(torch.isfinite(one).all()) and bool((one[1] == 0).all())
