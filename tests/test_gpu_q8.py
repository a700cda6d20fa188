"""The 8-bit cache on the GPU: the cache write against the NumPy definition bit for
bit, decode attention against fp64 over the codes' values.

Tolerance of the attention (derived, elementwise): the softmax weights (V scale
included) are rounded to fp16 for the product with V, at most 2^-11 of
themselves, or 2^-25 of the largest weight below fp16's normal range (the
running maximum is reached by one token, so that weight is at least 1 in the
kernel's units); scores and exponents are fp32: with |x| log2 units of magnitude
an exponent is off by at most 2^-22 |x| (product of K scale and softmax scale,
the multiplication, the sum with log2 of the V scale, the difference to the
maximum), the hardware exp2 and log2 add 2^-21; the same factor enters the
denominator.  fp32 sums of n terms add n 2^-24.  The result is rounded to fp16
once: 2^-11 of itself, or 2^-25 where it is subnormal.
"""
import numpy as np
import pytest
import torch

from oracle import q8 as oq
from paged_kv_cache_138_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
D = 128
SCALE = 1.0 / np.sqrt(D)
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def codes_to_dev(codes, code):
    if code == "int8":
        return dev(codes.astype(np.int8))
    return dev(codes.astype(np.float32)).to(torch.float8_e4m3fn)


def codes_of(t, code):
    if code == "int8":
        return t.cpu().numpy().astype(np.float64)
    return oq.e4m3_bits_to_value(t.view(torch.uint8).cpu().numpy())


def packed(rng, new, Hkv, behind=0, spread=True):
    """Packed fp16 rows whose magnitudes differ between tokens."""
    T = int(np.sum(new)) + behind
    x = rng.standard_normal((T, Hkv, D))
    if spread:
        x *= np.exp2(rng.integers(-3, 4, size=(T, 1, 1)))
    return x.astype(np.float16)


def starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def batch(rng, lens, bs, extra=3, pad=-1):
    nb = sum(wl.blocks_for(max(int(L), 1), bs) for L in lens) + extra
    tables = wl.handout_tables([max(int(L), 1) for L in lens], rng.permutation(nb).astype(np.int32),
                               bs, pad=pad)
    return nb, tables


def tolerance(ref, spread, peak, top, lens):
    n = np.asarray(lens, np.float64)[:, None, None]
    x = top[:, :, None] * 1.4427
    rel = 2.0 ** -11 + 2 * (2.0 ** -22 * (x + 48) + 2.0 ** -21) + 2 * n * 2.0 ** -24
    return (2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + rel * spread * 1.01 +
            n * 2.0 ** -25 * 448 * peak[:, :, None])


# ---- the cache write ---------------------------------------------------------------

@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("new,cached,Hkv", [
    ([1, 1, 1, 1], [0, 7, 16, 31], 8),          # single tokens: fresh, inside, first of a block
    ([5, 0, 17, 64, 1], [0, 9, 3, 0, 200], 1),  # ragged, a sequence that brings nothing
    ([130, 1, 33], [15, 64, 1], 5),             # odd head count
    ([300], [0], 2),
])
def test_write_matches_definition(ops, code, bs, new, cached, Hkv):
    rng = np.random.default_rng([bs, Hkv, len(new)])
    lens = (np.array(new) + np.array(cached)).astype(np.int32)
    nb, tables = batch(rng, lens, bs)
    qs = starts(new)
    x = {n: packed(rng, new, Hkv, behind=3) for n in "kv"}
    # earlier rows, and rows that hold nothing: any code, any scale
    codes = {n: oq.nearest_code(rng.standard_normal((nb, bs, Hkv, D)) * 40, code) for n in "kv"}
    stride = -(-Hkv // 4) * 4
    scales = {n: (np.abs(rng.standard_normal((nb, stride))) * 0.02).astype(np.float32) for n in "kv"}
    t = {n: codes_to_dev(codes[n], code) for n in "kv"}
    sc = {n: dev(scales[n]) for n in "kv"}
    err = ops.new_error_word()
    ops.reshape_and_cache_q8(dev(x["k"]), dev(x["v"]), dev(qs), dev(tables), dev(lens), t["k"],
                             t["v"], sc["k"], sc["v"], dev_err=err)
    assert ops.read_error_word(err) == 0
    for n in "kv":
        oq.write(x[n], qs, tables, lens, codes[n], scales[n], bs, code)
        assert np.array_equal(sc[n].cpu().numpy(), scales[n])
        assert np.array_equal(codes_of(t[n], code), codes[n])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_write_token_by_token(ops, code):
    """70 decode steps into one block table: the scale grows, earlier rows follow."""
    rng = np.random.default_rng(5)
    Hkv, bs = 4, 16
    nb, tables = batch(rng, [70, 70], bs)
    kc, vc, ks, vs = ops.q8_cache(nb, Hkv, bs, DTYPE[code])
    codes = [np.zeros((nb, bs, Hkv, D)) for _ in "kv"]
    scales = [np.zeros((nb, 4), np.float32) for _ in "kv"]
    qs = starts([1, 1])
    err = ops.new_error_word()
    for step in range(70):
        lens = np.array([step + 1, max(step, 1)], np.int32)
        x = [packed(rng, [1, 1], Hkv) for _ in "kv"]
        ops.reshape_and_cache_q8(dev(x[0]), dev(x[1]), dev(qs), dev(tables), dev(lens), kc, vc, ks,
                                 vs, dev_err=err)
        for i in range(2):
            oq.write(x[i], qs, tables, lens, codes[i], scales[i], bs, code)
    assert ops.read_error_word(err) == 0
    for i, (c, s) in enumerate(((kc, ks), (vc, vs))):
        assert np.array_equal(s.cpu().numpy(), scales[i])
        assert np.array_equal(codes_of(c, code), codes[i])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_write_extremes(ops, code):
    """Zeros, the least subnormal, the largest fp16, and values that are not finite."""
    rng = np.random.default_rng(6)
    Hkv, bs = 2, 16
    x = np.zeros((64, Hkv, D), np.float16)
    x[16:32] = np.float16(2 ** -24)
    x[32:48] = rng.choice([-65504, 65504, 1], size=(16, Hkv, D)).astype(np.float16)
    x[48:64] = rng.standard_normal((16, Hkv, D)).astype(np.float16)
    x[50, 0, 3], x[51, 0, 4], x[52, 1, 5] = np.inf, -np.inf, np.nan
    x[53, 1] = np.nan
    tables, lens, qs = np.array([[2, 0, 3, 1]], np.int32), np.array([64], np.int32), starts([64])
    kc, vc, ks, vs = ops.q8_cache(4, Hkv, bs, DTYPE[code])
    err = ops.new_error_word()
    ops.reshape_and_cache_q8(dev(x), dev(x), dev(qs), dev(tables), dev(lens), kc, vc, ks, vs,
                             dev_err=err)
    assert ops.read_error_word(err) == 8    # PKV_DEV_NONFINITE
    codes, scales = np.zeros((4, bs, Hkv, D)), np.zeros((4, 4), np.float32)
    oq.write(x, qs, tables, lens, codes, scales, bs, code)
    assert np.array_equal(ks.cpu().numpy(), scales) and np.array_equal(vs.cpu().numpy(), scales)
    assert np.array_equal(codes_of(kc, code), codes) and np.array_equal(codes_of(vc, code), codes)


def test_write_bad_metadata_is_reported_and_left_out(ops):
    rng = np.random.default_rng(7)
    Hkv, bs = 4, 16
    new = [20, 20, 20]
    x = dev(packed(rng, new, Hkv))
    lens = np.array([20, 20, 20], np.int32)
    good = np.array([[0, 1], [2, 3], [4, 5]], np.int32)

    def run(tables=good, lens=lens, qs=starts(new), x=x):
        kc, vc, ks, vs = ops.q8_cache(6, Hkv, bs)
        err = ops.new_error_word()
        ops.reshape_and_cache_q8(x, x, dev(np.asarray(qs, np.int32)), dev(tables), dev(lens), kc,
                                 vc, ks, vs, dev_err=err)
        return ops.read_error_word(err), ks.cpu().numpy()[:, :Hkv] > 0

    code, wrote = run()
    assert code == 0 and wrote.all()
    for bad in (-1, 6, 2 ** 31 - 1):
        t = good.copy()
        t[1, 1] = bad
        code, wrote = run(tables=t)
        assert code == 1 and not wrote[3].any() and wrote[[0, 1, 2, 4, 5]].all()
    for n in (-5, 19, 33, 2 ** 31 - 1):     # negative, shorter than its rows, past the table
        code, wrote = run(lens=np.array([20, n, 20], np.int32))
        assert code == 2 and not wrote[[2, 3]].any() and wrote[[0, 1, 4, 5]].all()
    code, wrote = run(qs=[0, 20, 10, 60], lens=np.array([20, 20, 50], np.int32))
    assert code == 7 and not wrote[[2, 3]].any()
    code, wrote = run(qs=[0, 20, 40, 61])
    assert code == 7 and not wrote[[4, 5]].any() and wrote[:4].all()
    code, wrote = run(qs=[-3, 20, 40, 60])
    assert code == 7 and not wrote[[0, 1]].any() and wrote[2:].all()


# ---- decode attention -----------------------------------------------------------------

def decode_case(seed, lens, Hq, Hkv, bs, code, spread=0, garbage=True):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    nb, tables = batch(rng, lens, bs, pad=-7)
    q = wl.host_normal_fp16(rng, (len(lens), Hq, D))
    codes = [oq.nearest_code(rng.standard_normal((nb, bs, Hkv, D)) * oq.QMAX[code] / 4, code)
             for _ in "kv"]
    scales = [(np.exp2(rng.uniform(-spread, spread, (nb, Hkv))) * 4 / oq.QMAX[code])
              .astype(np.float32) for _ in "kv"]
    return q, codes, scales, tables, lens


def poison(tensors, scales, tables, lens, bs):
    """Every byte that no context holds is 0x7f (NaN in e4m3), such blocks' scales NaN."""
    t = [c.view(torch.uint8) for c in tensors]
    held = np.zeros((t[0].shape[0], bs), bool)
    for s, L in enumerate(lens):
        pos = np.arange(int(L))
        held[tables[s][pos // bs], pos % bs] = True
    free = dev(~held)
    for c in t:
        c[free] = 0x7f
    for s in scales:
        s[dev(~held.any(1))] = float("nan")


def run_decode(ops, q, codes, scales, tables, lens, code, bs, scale=SCALE, clean=False):
    t = [codes_to_dev(c, code) for c in codes]
    sc = [dev(s) for s in scales]
    if not clean:
        poison(t, sc, tables, lens, bs)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    err = ops.new_error_word()
    ops.paged_attention_decode_q8(out, dev(q), t[0], t[1], sc[0], sc[1], dev(tables), dev(lens),
                                  scale, dev_err=err)
    return out.cpu().numpy().astype(np.float64), ops.read_error_word(err)


def check_decode(got, q, codes, scales, tables, lens, bs, scale=SCALE):
    ref, spread, peak, top = oq.decode(q, codes[0], codes[1], scales[0], scales[1], tables, lens,
                                       scale, bs)
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - tolerance(ref, spread, peak, top, lens)
    assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 4), (16, 4), (16, 2), (5, 5)])
def test_decode_matches_oracle(ops, code, bs, Hq, Hkv):
    lens = [1, 0, 7, 8, 9, 31, 32, 33, 127, 129, 515]
    q, codes, scales, tables, lens = decode_case(bs * 100 + Hq + Hkv, lens, Hq, Hkv, bs, code)
    got, err = run_decode(ops, q, codes, scales, tables, lens, code, bs)
    assert err == 0
    assert (got[1] == 0).all()
    check_decode(got, q, codes, scales, tables, lens, bs)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("bs", [8, 16, 64])
def test_decode_long_and_split(ops, code, bs):
    """Several splits of every length; block scales that differ by up to 2^24."""
    lens = [2500, 512, 513, 1, 5000, 2049]
    q, codes, scales, tables, lens = decode_case(bs, lens, 8, 2, bs, code, spread=12)
    # scores of a model's size: the scales above multiply K as well
    scales[0] = (np.abs(np.random.default_rng(1).standard_normal(scales[0].shape)) * 4 /
                 oq.QMAX[code]).astype(np.float32)
    got, err = run_decode(ops, q, codes, scales, tables, lens, code, bs)
    assert err == 0
    check_decode(got, q, codes, scales, tables, lens, bs)


@pytest.mark.parametrize("longest", [1000, 3584, 3600, 4096, 8700, 40000])
def test_decode_merges(ops, longest):
    """2, 7, 8, 9, 17 and 79 splits beside sequences of fewer and of none: rows merged by
    one warp and by a CTA."""
    lens = [longest, 1, 513, 0, longest // 2, longest - 1]
    q, codes, scales, tables, lens = decode_case(longest, lens, 8, 2, 16, "int8")
    got, err = run_decode(ops, q, codes, scales, tables, lens, "int8", 16)
    assert err == 0 and (got[3] == 0).all()
    check_decode(got, q, codes, scales, tables, lens, 16)


def test_decode_tiny_weights_on_large_scales(ops):
    """The tokens that carry the weight lie in blocks of tiny V scale; blocks of huge V
    scale have weights near 2^-60.  Zero scales among them."""
    rng = np.random.default_rng(3)
    q, codes, scales, tables, lens = decode_case(9, [200, 700], 8, 8, 16, "int8")
    q[:] = 0
    q[:, :, 0] = 1
    codes[0][:] = 0
    codes[0][..., 0] = -127
    light = tables[0, 3], tables[1, 20]
    codes[0][list(light), :, :, 0] = 127
    scales[0][:] = 21.0 / (127 * SCALE * 1.4427)       # +-21 log2 units ...
    scales[1][:] = 300.0
    scales[1][list(light)] = 1e-7
    scales[1][tables[1, 5]] = 0
    scales[1][tables[1, 21]] = 0
    got, err = run_decode(ops, q, codes, scales, tables, lens, "int8", 16)
    assert err == 0
    check_decode(got, q, codes, scales, tables, lens, 16)
    assert rng is not None


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_decode_dominant_keys_everywhere(ops, code):
    """One dominant key at a place of its own in every sequence: its V row comes back."""
    lens = [300] * 40
    q, codes, scales, tables, lens = decode_case(21, lens, 8, 8, 16, code)
    for s in range(40):
        pos = (s * 37) % 300
        b, r = tables[s, pos // 16], pos % 16
        for h in range(8):
            qq = q[s, h].astype(np.float64)
            codes[0][b, r, h] = oq.nearest_code(qq / np.abs(qq).max() * oq.QMAX[code], code)
        scales[0][b] = 0.5 / (1 if code == "int8" else 3.5)
    got, err = run_decode(ops, q, codes, scales, tables, lens, code, 16)
    assert err == 0
    check_decode(got, q, codes, scales, tables, lens, 16)


def test_decode_bad_metadata(ops):
    q, codes, scales, tables, lens = decode_case(4, [100, 40, 64], 8, 2, 16, "e4m3")
    t = tables.copy()
    t[0, 2], t[2, 0] = 10 ** 6, -1
    got, err = run_decode(ops, q, codes, scales, t, lens, "e4m3", 16, clean=True)
    assert err == 1
    # the tokens of the bad blocks are left out, the others attended
    keep = [np.r_[0:32, 48:100], np.arange(40), np.arange(16, 64)]
    for s in range(3):
        pos = keep[s]
        blk = tables[s][pos // 16]
        sub = [c[blk, pos % 16][:, None] for c in codes]
        ss = [x[blk] for x in scales]
        check_decode(got[s:s + 1], q[s:s + 1], sub, ss, np.arange(len(pos))[None],
                     np.array([len(pos)]), 1)
    bad = lens.copy()
    bad[1] = -4
    got, err = run_decode(ops, q, codes, scales, tables, bad, "e4m3", 16, clean=True)
    assert err == 2 and (got[1] == 0).all()


def test_decode_every_block_bad(ops):
    q, codes, scales, tables, lens = decode_case(4, [100, 600], 8, 2, 16, "int8")
    got, err = run_decode(ops, q, codes, scales, np.full_like(tables, -1), lens, "int8", 16,
                          clean=True)
    assert err == 1 and (got == 0).all()


def test_decode_same_bits_whatever_the_placement(ops):
    """Block ids, batch order and repeated launches leave the bits alone."""
    q, codes, scales, tables, lens = decode_case(8, [700, 33, 1500], 16, 4, 16, "int8")
    a, _ = run_decode(ops, q, codes, scales, tables, lens, "int8", 16)
    b, _ = run_decode(ops, q, codes, scales, tables, lens, "int8", 16)
    assert np.array_equal(a, b)
    perm = np.random.default_rng(0).permutation(codes[0].shape[0])
    inv = np.argsort(perm)
    moved = np.where(tables >= 0, inv[np.maximum(tables, 0)], tables).astype(np.int32)
    order = [2, 0, 1]
    c, _ = run_decode(ops, q[order], [x[perm] for x in codes], [x[perm] for x in scales],
                      moved[order], lens[order], "int8", 16)
    assert np.array_equal(a[order], c)


def test_graph_and_streams(ops):
    """Write and attention captured together and replayed on new tokens, then on
    another stream with a workspace of its own."""
    rng = np.random.default_rng(12)
    Hq, Hkv, bs = 8, 2, 16
    nb, tables = batch(rng, [600, 90], bs)
    kc, vc, ks, vs = ops.q8_cache(nb, Hkv, bs)
    codes = [np.zeros((nb, bs, Hkv, D)) for _ in "kv"]
    scales = [np.zeros((nb, 4), np.float32) for _ in "kv"]
    new = [580, 70]
    x = [packed(rng, new, Hkv, spread=False) for _ in "kv"]
    lens = np.array(new, np.int32)
    td, ld = dev(tables), dev(lens)
    ops.reshape_and_cache_q8(dev(x[0]), dev(x[1]), dev(starts(new)), td, ld, kc, vc, ks, vs)
    for i in range(2):
        oq.write(x[i], starts(new), tables, lens, codes[i], scales[i], bs, "int8")
    one = dev(starts([1, 1]))
    q = dev(wl.host_normal_fp16(rng, (2, Hq, D)))
    k1, v1 = dev(packed(rng, [1, 1], Hkv)), dev(packed(rng, [1, 1], Hkv))
    out, err = torch.zeros_like(q), ops.new_error_word()
    ws = ops.alloc_workspace(2, Hq, tables.shape[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.reshape_and_cache_q8(k1, v1, one, td, ld, kc, vc, ks, vs, dev_err=err)
        ops.paged_attention_decode_q8(out, q, kc, vc, ks, vs, td, ld, SCALE, workspace=ws,
                                      dev_err=err)
    for step in range(20):
        lens = lens + 1
        ld.copy_(dev(lens))
        for i, t in enumerate((k1, v1)):
            x = packed(rng, [1, 1], Hkv)
            t.copy_(dev(x))
            oq.write(x, starts([1, 1]), tables, lens, codes[i], scales[i], bs, "int8")
        graph.replay()
    assert ops.read_error_word(err) == 0
    assert np.array_equal(codes_of(kc, "int8"), codes[0])
    got = out.cpu().numpy().astype(np.float64)
    check_decode(got, q.cpu().numpy(), codes, scales, tables, lens, bs)
    side = torch.cuda.Stream()
    out2 = torch.zeros_like(q)
    torch.cuda.synchronize()
    launch = ops.paged_attention_decode_q8(out2, q, kc, vc, ks, vs, td, ld, SCALE, stream=side,
                                           prepare=True)
    launch()
    side.synchronize()
    assert torch.equal(out, out2)


def test_copy_blocks_moves_codes_and_scales(ops):
    """Copy-on-write of an 8-bit block with the cache's own copy_blocks."""
    rng = np.random.default_rng(2)
    for Hkv in (1, 2, 8):
        kc, vc, ks, vs = ops.q8_cache(6, Hkv, 16, torch.float8_e4m3fn)
        for t in (kc, vc):
            t.view(torch.uint8).copy_(dev(rng.integers(0, 120, size=tuple(t.shape)).astype(np.uint8)))
        for t in (ks, vs):
            t.copy_(dev(rng.standard_normal(tuple(t.shape)).astype(np.float32)))
        pairs = dev(np.array([[1, 4], [2, 0]], np.int64))
        want = [t.clone() for t in (kc, vc, ks, vs)]
        for t in want:
            u = t.view(torch.uint8)
            u[4], u[0] = u[1].clone(), u[2].clone()
        ops.copy_blocks(kc, vc, pairs)
        ops.copy_blocks(ks, vs, pairs)
        for a, b in zip((kc, vc, ks, vs), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_wrappers_refuse(ops):
    kc, vc, ks, vs = ops.q8_cache(8, 2, 16)
    q = torch.zeros((2, 4, D), dtype=torch.float16, device="cuda")
    k = torch.zeros((2, 2, D), dtype=torch.float16, device="cuda")
    t = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        ops.q8_cache(8, 2, 16, torch.float16)
    with pytest.raises(TypeError):
        ops.paged_attention_decode_q8(q, q, kc.half(), vc, ks, vs, t, n, 1.0)
    with pytest.raises(TypeError):
        ops.paged_attention_decode_q8(q, q, kc, vc.view(torch.float8_e4m3fn), ks, vs, t, n, 1.0)
    with pytest.raises(ValueError):
        ops.paged_attention_decode_q8(q, q, kc, vc, ks[:, :1].contiguous(), vs[:, :1].contiguous(),
                                      t, n, 1.0)
    with pytest.raises(ValueError):
        ops.paged_attention_decode_q8(q, q, kc, vc, ks[:, ::2], vs, t, n, 1.0)
    with pytest.raises(ValueError):
        ops.reshape_and_cache_q8(k, k, qs[:2], t, n, kc, vc, ks, vs)
    with pytest.raises(TypeError):
        ops.reshape_and_cache_q8(k, k, qs.long(), t, n, kc, vc, ks, vs)
    with pytest.raises(ValueError):
        ops.reshape_and_cache_q8(k[:, :1], k[:, :1], qs, t, n, kc, vc, ks, vs)
    with pytest.raises(TypeError):
        ops.reshape_and_cache_q8(k.cpu(), k, qs, t, n, kc, vc, ks, vs)
