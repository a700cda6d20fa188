"""Rotary positions on the GPU, alone and with the cache writes, against the NumPy definition
bit for bit: the rotation is four products and two sums in fp32 in a fixed order, so the fp16
results and the 8-bit codes have one right value each."""
import numpy as np
import pytest
import torch

from oracle import q8 as oq
from oracle import rope as orope
from paged_kv_cache_138_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
D = 128
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(a):
    return np.ascontiguousarray(a, dtype=np.float16).view(np.uint16)


def codes_to_dev(codes, code):
    if code == "int8":
        return dev(codes.astype(np.int8))
    return dev(codes.astype(np.float32)).to(torch.float8_e4m3fn)


def codes_of(t, code):
    if code == "int8":
        return t.cpu().numpy().astype(np.float64)
    return oq.e4m3_bits_to_value(t.view(torch.uint8).cpu().numpy())


def table_of(n, rows, seed=0):
    f = 10000.0 ** (-np.arange(n) / n)
    return orope.table64(f, rows, 1.0 + 0.1 * seed).astype(np.float32)


def projection(rng, T, Hq, Hkv):
    """q, k and v as slices of one output, tokens of different sizes."""
    x = (rng.standard_normal((T, Hq + 2 * Hkv, D)) *
         np.exp2(rng.integers(-3, 4, size=(T, 1, 1)))).astype(np.float16)
    t = dev(x)
    cut = lambda a: (a[:, :Hq], a[:, Hq:Hq + Hkv], a[:, Hq + Hkv:])   # noqa: E731
    return cut(x), cut(t)


def axes_of(n, num_axes, rng):
    return None if num_axes == 1 else tuple(int(a) for a in rng.integers(0, num_axes, n))


def starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def batch(rng, lens, bs, extra=3):
    nb = sum(wl.blocks_for(max(int(L), 1), bs) for L in lens) + extra
    order = rng.permutation(nb).astype(np.int32)
    return nb, wl.handout_tables([max(int(L), 1) for L in lens], order, bs, pad=-1)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("rot,num_axes", [(128, 1), (128, 3), (96, 2), (64, 1), (16, 4), (112, 1)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (7, 8, 2), (33, 5, 3), (130, 32, 8), (2, 40, 40)])
def test_rotary(ops, T, Hq, Hkv, rot, num_axes, adjacent):
    rng = np.random.default_rng([T, rot, num_axes])
    (q, k, _), (tq, tk, _) = projection(rng, T, Hq, Hkv)
    table = table_of(rot // 2, 500)
    pos = rng.integers(0, 500, (num_axes, T)).astype(np.int32)
    pos[:, 0], pos[:, -1] = 0, 499
    axes = axes_of(rot // 2, num_axes, rng)
    err = ops.new_error_word()
    qo, ko = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda"), torch.empty(
        (T, Hkv, D), dtype=torch.float16, device="cuda")
    tpos = dev(pos if num_axes > 1 else pos[0])
    ops.rotary_embedding(qo, ko, tq, tk, tpos, dev(table), axes=axes, adjacent=adjacent, dev_err=err)
    for x, y in ((q, qo), (k, ko)):
        assert np.array_equal(bits(y.cpu().numpy()),
                              bits(orope.rotate(x, pos, table, axes, adjacent)))
    # in place, in the slices themselves; then q alone
    want = [t.clone() for t in (qo, ko)]
    ops.rotary_embedding(tq, tk, tq, tk, tpos, dev(table), axes=axes, adjacent=adjacent, dev_err=err)
    assert torch.equal(tq, want[0]) and torch.equal(tk, want[1])
    ops.rotary_embedding(qo, None, tq, None, tpos, dev(table), axes=axes, adjacent=adjacent,
                         dev_err=err)
    assert np.array_equal(bits(qo.cpu().numpy()), bits(orope.rotate(
        want[0].cpu().numpy(), pos, table, axes, adjacent)))
    assert ops.read_error_word(err) == 0


def test_rotary_leaves_out_bad_positions(ops):
    rng = np.random.default_rng(3)
    (q, k, _), (tq, tk, _) = projection(rng, 6, 8, 2)
    table = table_of(64, 50)
    pos = rng.integers(0, 50, (2, 6)).astype(np.int32)
    pos[0, 1], pos[1, 4] = 50, -1
    axes = axes_of(64, 2, rng)
    err = ops.new_error_word()
    qo, ko = torch.full((6, 8, D), 7.0, dtype=torch.float16, device="cuda"), torch.full(
        (6, 2, D), 7.0, dtype=torch.float16, device="cuda")
    ops.rotary_embedding(qo, ko, tq, tk, dev(pos), dev(table), axes=axes, dev_err=err)
    assert ops.read_error_word(err) == 5
    good = [0, 2, 3, 5]
    for x, y in ((q, qo), (k, ko)):
        y = y.cpu().numpy()
        ref = orope.rotate(x[good], pos[:, good], table, axes)
        assert np.array_equal(bits(y[good]), bits(ref)) and (y[[1, 4]] == 7).all()
    ops.rotary_embedding(qo, ko, tq, tk, dev(pos), dev(table), axes=axes)      # without a word
    ops.rotary_embedding(qo[:0], ko[:0], tq[:0], tk[:0], dev(pos)[:, :0].contiguous(), dev(table),
                         axes=axes)


def test_table_of_far_positions(ops):
    f = 10000.0 ** (-np.arange(64) / 64)
    t = ops.rope_table(f, (1 << 20) + 5, magnitude=0.5)
    at = [0, 1, 65535, 65536, 1 << 20, (1 << 20) + 4]
    angle = np.array(at, np.float64)[:, None] * f
    ref = 0.5 * np.stack([np.cos(angle), np.sin(angle)], axis=-1)
    assert np.abs(t[at].cpu().numpy() - ref).max() <= 0.5 * 2.0 ** -24 + 1e-9


CASES = [
    ([1, 1, 1, 1], [0, 7, 16, 31], 8, 8),             # a step's single tokens
    ([1, 2, 0, 3, 1, 17], [0, 15, 3, 15, 64, 30], 40, 5),   # few tokens: pieces of several rows
    ([5, 0, 17, 64, 1], [0, 9, 3, 0, 200], 8, 1),     # ragged, a sequence that brings nothing
    ([130, 1, 33], [15, 64, 1], 12, 3),               # odd head counts
    ([300], [0], 32, 8),
]


@pytest.mark.parametrize("bs", [1, 5, 16, 64])
@pytest.mark.parametrize("new,cached,Hq,Hkv", CASES)
def test_append(ops, bs, new, cached, Hq, Hkv):
    rng = np.random.default_rng([bs, Hkv, len(new)])
    lens = (np.array(new) + np.array(cached)).astype(np.int32)
    nb, tables = batch(rng, lens, bs)
    qs, T = starts(new), int(np.sum(new)) + 3          # 3 rows that no sequence owns
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    num_axes, adjacent, rot = 1 + 2 * (bs & 1), bool(Hkv & 1), 64 if bs == 5 else 128
    table, axes = table_of(rot // 2, 1000), axes_of(rot // 2, num_axes, rng)
    seq, place = orope.places(qs, lens, T)
    pos = place[None] if num_axes == 1 else rng.integers(0, 1000, (num_axes, T)).astype(np.int32)
    kc = rng.standard_normal((nb, bs, Hkv, D)).astype(np.float16)
    vc = rng.standard_normal((nb, bs, Hkv, D)).astype(np.float16)
    dk, dv = dev(kc), dev(vc)
    qo = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    err = ops.new_error_word()
    ops.rope_and_cache(qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), dk, dv, dev(table),
                       positions=None if num_axes == 1 else dev(pos), axes=axes, adjacent=adjacent,
                       dev_err=err)
    assert ops.read_error_word(err) == 0
    own = T - 3
    ref_q = orope.rotate(q[:own], pos[:, :own], table, axes, adjacent)
    ref_k = orope.rotate(k[:own], pos[:, :own], table, axes, adjacent)
    at = tables[seq[:own], place[:own] // bs], place[:own] % bs
    kc[at], vc[at] = ref_k.astype(np.float16), v[:own]
    assert np.array_equal(bits(dk.cpu().numpy()), bits(kc))
    assert np.array_equal(bits(dv.cpu().numpy()), bits(vc))
    qo = qo.cpu().numpy()
    assert np.array_equal(bits(qo[:own]), bits(ref_q)) and (qo[own:] == 7).all()
    # in two steps: rotated in place, then scattered by slots: the same bits
    if bs == 16:
        dk2, dv2 = dev(kc * 0), dev(vc * 0)
        slots = np.where(seq >= 0, 0, -1).astype(np.int64)
        slots[:own] = at[0].astype(np.int64) * bs + at[1]
        ops.rotary_embedding(tq, tk, tq, tk, dev(np.maximum(pos[0], 0).astype(np.int32)), dev(table),
                             adjacent=adjacent)
        ops.reshape_and_cache(tk.contiguous(), tv.contiguous(), dev(slots), dk2, dv2)
        assert torch.equal(dk2[dev(at[0]).long(), dev(at[1]).long()],
                           dk[dev(at[0]).long(), dev(at[1]).long()])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("new,cached,Hq,Hkv", CASES)
def test_append_q8(ops, code, bs, new, cached, Hq, Hkv):
    rng = np.random.default_rng([bs, Hkv, len(new)])
    lens = (np.array(new) + np.array(cached)).astype(np.int32)
    nb, tables = batch(rng, lens, bs)
    qs, T = starts(new), int(np.sum(new)) + 3
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    num_axes, adjacent, rot = (3, True, 128) if bs == 16 else (1, bs == 64, 96 if bs == 8 else 128)
    table, axes = table_of(rot // 2, 1000, seed=1), axes_of(rot // 2, num_axes, rng)
    seq, place = orope.places(qs, lens, T)
    pos = place[None] if num_axes == 1 else rng.integers(0, 1000, (num_axes, T)).astype(np.int32)
    stride = -(-Hkv // 4) * 4
    codes = {n: oq.nearest_code(rng.standard_normal((nb, bs, Hkv, D)) * 40, code) for n in "kv"}
    scales = {n: (np.abs(rng.standard_normal((nb, stride))) * 0.02).astype(np.float32) for n in "kv"}
    t = {n: codes_to_dev(codes[n], code) for n in "kv"}
    sc = {n: dev(scales[n]) for n in "kv"}
    qo = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    err = ops.new_error_word()
    args = (qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), t["k"], t["v"], sc["k"], sc["v"],
            dev(table))
    more = dict(positions=None if num_axes == 1 else dev(pos), axes=axes, adjacent=adjacent,
                dev_err=err)
    ops.rope_and_cache_q8(*args, **more)
    assert ops.read_error_word(err) == 0
    own = T - 3
    x = {"k": orope.rotate(k[:own], pos[:, :own], table, axes, adjacent), "v": v[:own]}
    for n in "kv":
        oq.write(x[n], qs, tables, lens, codes[n], scales[n], bs, code)
        assert np.array_equal(sc[n].cpu().numpy(), scales[n])
        assert np.array_equal(codes_of(t[n], code), codes[n])
    got = qo.cpu().numpy()
    assert np.array_equal(bits(got[:own]), bits(orope.rotate(q[:own], pos[:, :own], table, axes, adjacent)))
    assert (got[own:] == 7).all()
    # the same tokens again: nothing changes (no scale grows)
    before = [a.clone() for a in (t["k"].view(torch.uint8), t["v"].view(torch.uint8), sc["k"], sc["v"])]
    ops.rope_and_cache_q8(*args, **more)
    after = (t["k"].view(torch.uint8), t["v"].view(torch.uint8), sc["k"], sc["v"])
    assert all(torch.equal(a, b) for a, b in zip(before, after))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1], [40, 3, 1, 9, 2]])
def test_q8_step_after_step(ops, code, new):
    """Tokens that grow a block's scale, one call after another, by both ways of cutting."""
    rng = np.random.default_rng(len(new))
    S, Hq, Hkv, bs = len(new), 8, 2, 16
    lens = np.array([3, 15, 16, 30, 1])
    nb, tables = batch(rng, lens + 4 * np.array(new), bs)
    table = table_of(64, 500)
    codes = {n: np.zeros((nb, bs, Hkv, D)) for n in "kv"}
    scales = {n: np.zeros((nb, 4), np.float32) for n in "kv"}
    cache = ops.q8_cache(nb, Hkv, bs, dtype=DTYPE[code])
    err = ops.new_error_word()
    held = np.zeros(S, int)
    for step in range(4):
        n_now = lens if step == 0 else np.array(new)
        held = held + n_now
        (q, k, v), (tq, tk, tv) = projection(rng, int(n_now.sum()), Hq, Hkv)
        qs = starts(n_now)
        qo = torch.empty((int(n_now.sum()), Hq, D), dtype=torch.float16, device="cuda")
        ops.rope_and_cache_q8(qo, tq, tk, tv, dev(qs), dev(tables), dev(held.astype(np.int32)),
                              *cache, dev(table), dev_err=err)
        _, place = orope.places(qs, held, len(q))
        for n, x in (("k", orope.rotate(k, place, table)), ("v", v)):
            oq.write(x, qs, tables, held, codes[n], scales[n], bs, code)
    assert ops.read_error_word(err) == 0
    for n, c, s in (("k", cache[0], cache[2]), ("v", cache[1], cache[3])):
        assert np.array_equal(s.cpu().numpy(), scales[n]) and np.array_equal(codes_of(c, code), codes[n])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("new,cached", [
    ([1] * 40 + [70] + [1] * 9, [11 * i % 130 for i in range(50)]),      # a chunk among single tokens
    ([4, 9, 15, 5, 31], [3, 60, 1, 0, 40]),           # pieces that share their heads, ends of blocks
    ([30, 1, 0, 25, 64], [0, 64, 5, 63, 0]),          # whole blocks
])
def test_q8_long_pieces_of_steps(ops, code, bs, new, cached):
    """Several rows of a block in a call of few tokens a sequence, a token off the table
    and values that are not finite among them."""
    rng = np.random.default_rng([bs, len(new)])
    Hq, Hkv, rows = 13, 3, 200
    lens = (np.array(new) + np.array(cached)).astype(np.int32)
    nb, tables = batch(rng, lens, bs)
    qs, T = starts(new), int(np.sum(new))
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    table, axes = table_of(64, rows, seed=2), axes_of(64, 3, rng)
    pos = rng.integers(0, rows, (3, T)).astype(np.int32)
    seq, place = orope.places(qs, lens, T)
    s_long = int(np.argmax(new))
    out, bad = int(qs[s_long]) + 2, int(qs[s_long]) + 3
    k, v = k.copy(), v.copy()
    k[bad, 1, 40], v[bad, 2, 7] = np.inf, np.nan
    tk, tv = dev(k), dev(v)
    codes = {n: oq.nearest_code(rng.standard_normal((nb, bs, Hkv, D)) * 40, code) for n in "kv"}
    scales = {n: (np.abs(rng.standard_normal((nb, 4))) * 0.02).astype(np.float32) for n in "kv"}
    with np.errstate(invalid="ignore"):
        x = {"k": orope.rotate(k, pos, table, axes), "v": v.astype(np.float32)}

    def call(pos):
        t = {n: codes_to_dev(codes[n], code) for n in "kv"}
        sc = {n: dev(scales[n]) for n in "kv"}
        qo = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
        err = ops.new_error_word()
        ops.rope_and_cache_q8(qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), t["k"], t["v"],
                              sc["k"], sc["v"], dev(table), positions=dev(pos), axes=axes, dev_err=err)
        return qo.cpu().numpy(), t, sc, ops.read_error_word(err)

    qo, t, sc, err = call(pos)
    assert err == 8
    want = {n: (codes[n].copy(), scales[n].copy()) for n in "kv"}
    for n in "kv":
        oq.write(x[n], qs, tables, lens, *want[n], bs, code)
        assert np.array_equal(sc[n].cpu().numpy(), want[n][1])
        assert np.array_equal(codes_of(t[n], code), want[n][0])
    assert np.array_equal(bits(qo), bits(orope.rotate(q, pos, table, axes)))
    # a token off the table on one axis: its q and its codes as they were, all else as before
    off = pos.copy()
    off[2, out] = rows
    qo, t, sc, err = call(off)
    assert err in (5, 8) and (qo[out] == 7).all()
    keep = np.arange(T) != out
    assert np.array_equal(bits(qo[keep]), bits(orope.rotate(q, pos, table, axes)[keep]))
    blk, row = tables[s_long, place[out] // bs], place[out] % bs
    for n in "kv":
        y = x[n].copy()
        y[out] = 0
        c, s = codes[n].copy(), scales[n].copy()
        oq.write(y, qs, tables, lens, c, s, bs, code)
        got = codes_of(t[n], code)
        assert np.array_equal(sc[n].cpu().numpy(), s)
        assert np.array_equal(got[blk, row], codes[n][blk, row])
        got[blk, row] = c[blk, row]
        assert np.array_equal(got, c)


@pytest.mark.parametrize("bs", [8, 32])
@pytest.mark.parametrize("n", [1, 2, 7, 70])
def test_q8_left_out_tokens_start_a_block(ops, n, bs):
    """A block that held another sequence's tokens, whose new first tokens are all left out:
    its scale starts again, and the next token gets one of its own."""
    rng = np.random.default_rng(n)
    Hq, Hkv, rows = 4, 2, 50
    table = table_of(64, rows)
    nb = n // bs + 2
    tables = rng.permutation(nb).astype(np.int32)[None, :(n + 1 + bs - 1) // bs]
    (q, k, v), (tq, tk, tv) = projection(rng, n + 1, Hq, Hkv)
    pos = np.array([rows] * n + [3], np.int32)
    cache = ops.q8_cache(nb, Hkv, bs)
    cache[2].fill_(5.0), cache[3].fill_(5.0)
    err = ops.new_error_word()
    for a, b in ((0, n), (n, n + 1)):
        qo = torch.empty((b - a, Hq, D), dtype=torch.float16, device="cuda")
        ops.rope_and_cache_q8(qo, tq[a:b], tk[a:b], tv[a:b], dev(starts([b - a])), dev(tables),
                              dev(np.array([b], np.int32)), *cache, dev(table),
                              positions=dev(pos[a:b]), dev_err=err)
        assert ops.read_error_word(err) == 5
    blk = tables[0, n // bs]
    for x, c, s in ((orope.rotate(k[n:], pos[n:], table), cache[0], cache[2]),
                    (v[n:].astype(np.float32), cache[1], cache[3])):
        amax = np.abs(x[0]).max(axis=-1).astype(np.float32)
        assert np.array_equal(s[blk, :Hkv].cpu().numpy(), amax / np.float32(127))
        assert (codes_of(c, "int8")[tables[0], :].reshape(-1, Hkv, D)[:n] == 0).all()


@pytest.mark.parametrize("T,S", [(3, 3), (40, 3)])
def test_q8_not_finite_and_bad_metadata(ops, T, S):
    rng = np.random.default_rng(T)
    Hq, Hkv, bs, code = 8, 2, 16, "int8"
    new = [T // S + (T % S if s == 0 else 0) for s in range(S)]
    lens = np.array(new, np.int32)
    nb, tables = batch(rng, lens, bs)
    table, qs = table_of(64, 100), starts(new)
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    k, v = k.copy(), v.copy()
    k[0, 0, 3], k[T - 1, 1, 100], v[1, 1, 7] = np.inf, np.nan, -np.inf
    tk, tv = dev(k), dev(v)
    tables[S - 1, 0] = nb                      # the last sequence's first block does not exist
    _, place = orope.places(qs, lens, T)

    def call(**a):
        cache = ops.q8_cache(nb, Hkv, bs)
        err = ops.new_error_word()
        qo = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
        args = dict(qs=dev(qs), tables=dev(tables), lens=dev(lens), table=dev(table))
        args.update(a)
        ops.rope_and_cache_q8(qo, tq, tk, tv, args["qs"], args["tables"], args["lens"], *cache,
                              args["table"], dev_err=err)
        return qo.cpu().numpy(), cache, ops.read_error_word(err)

    qo, cache, code_got = call()
    assert code_got in (1, 8)
    with np.errstate(invalid="ignore"):
        x = {"k": orope.rotate(k, place, table), "v": v.astype(np.float32)}
    for n, c, s in (("k", cache[0], cache[2]), ("v", cache[1], cache[3])):
        codes, scales = np.zeros((nb + 1, bs, Hkv, D)), np.zeros((nb + 1, 4), np.float32)
        oq.write(x[n], qs, tables, lens, codes, scales, bs, code)
        assert np.array_equal(s.cpu().numpy(), scales[:nb]) and np.array_equal(codes_of(c, code), codes[:nb])
    assert np.array_equal(bits(qo), bits(orope.rotate(q, place, table)))       # q all the same
    # a table that ends early: those tokens are left out, their q as it was
    qo, cache, code_got = call(table=dev(table[:1]))
    assert code_got in (1, 5, 8) and (qo[place > 0] == 7).all()
    assert np.array_equal(bits(qo[place == 0]), bits(orope.rotate(q[place == 0], place[place == 0], table)))
    assert not codes_of(cache[0], code)[:, 1:].any()
    # lengths that do not hold the rows, and rows past the batch
    bad = lens.copy()
    bad[0] = new[0] - 1
    qo, cache, code_got = call(lens=dev(bad))
    assert code_got in (1, 2, 8) and (qo[:new[0]] == 7).all()
    late = qs.copy()
    late[S] = T + 1
    qo, cache, code_got = call(qs=dev(late))
    assert code_got in (1, 7, 8) and (qo[qs[S - 1]:] == 7).all()


def test_fp16_bad_metadata(ops):
    rng = np.random.default_rng(9)
    new, Hq, Hkv, bs = [5, 40, 2], 8, 2, 16
    lens, qs, T = np.array(new, np.int32), starts(new), 47
    nb, tables = batch(rng, lens, bs)
    table = table_of(64, 100)
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    _, place = orope.places(qs, lens, T)
    for kind, code in (("block", 1), ("len", 2), ("range", 7), ("table", 5)):
        t2, l2, q2, tab, gone = tables.copy(), lens.copy(), qs.copy(), table, np.zeros(T, bool)
        if kind == "block":
            t2[1, 1] = -5
        elif kind == "len":
            l2[1] = 1000
            gone[5:45] = True
        elif kind == "range":
            q2[3] = 48
            gone[45:] = True
        else:
            tab = table[:30]
            gone = place >= 30
        kc = torch.zeros((nb, bs, Hkv, D), dtype=torch.float16, device="cuda")
        vc, err = torch.zeros_like(kc), ops.new_error_word()
        qo = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
        ops.rope_and_cache(qo, tq, tk, tv, dev(q2), dev(t2), dev(l2), kc, vc, dev(tab), dev_err=err)
        assert ops.read_error_word(err) == code
        qo = qo.cpu().numpy()
        assert (qo[gone] == 7).all()
        assert np.array_equal(bits(qo[~gone]), bits(orope.rotate(q[~gone], place[~gone], table)))
        seq, _ = orope.places(qs, lens, T)
        ref = np.zeros((nb, bs, Hkv, D), np.float16)
        stored = ~gone & ~((seq == 1) & (place // bs == 1) & (kind == "block"))
        ref[tables[seq[stored], place[stored] // bs], place[stored] % bs] = v[stored]
        assert np.array_equal(bits(vc.cpu().numpy()), bits(ref))


def test_streams_and_graphs(ops):
    """On another stream than the current one, prepared, and captured and replayed on new values."""
    rng = np.random.default_rng(4)
    new, Hq, Hkv, bs = [1, 1, 1], 8, 2, 16
    lens, qs = np.array([5, 16, 17], np.int32), starts(new)
    nb, tables = batch(rng, lens, bs)
    table = table_of(64, 100)
    (q, k, v), (tq, tk, tv) = projection(rng, 3, Hq, Hkv)
    place = lens - 1
    kc = torch.zeros((nb, bs, Hkv, D), dtype=torch.float16, device="cuda")
    vc, cache = torch.zeros_like(kc), ops.q8_cache(nb, Hkv, bs)
    qo, qo8 = (torch.empty((3, Hq, D), dtype=torch.float16, device="cuda") for _ in range(2))
    dqs, dt, dl, dtab = dev(qs), dev(tables), dev(lens), dev(table)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls = [ops.rope_and_cache(qo, tq, tk, tv, dqs, dt, dl, kc, vc, dtab, stream=side, prepare=True),
             ops.rope_and_cache_q8(qo8, tq, tk, tv, dqs, dt, dl, *cache, dtab, stream=side,
                                   prepare=True)]
    for c in calls:
        c()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for c in calls:
            c()
    for round_ in range(2):
        if round_:
            (q, k, v), (t0, t1, t2) = projection(rng, 3, Hq, Hkv)
            for a, b in ((tq, t0), (tk, t1), (tv, t2)):
                a.copy_(b)
            for t in cache:
                t.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
        ref = bits(orope.rotate(q, place, table))
        assert np.array_equal(bits(qo.cpu().numpy()), ref) and np.array_equal(bits(qo8.cpu().numpy()), ref)
        at = tables[np.arange(3), place // bs], place % bs
        rk = orope.rotate(k, place, table)
        assert np.array_equal(bits(kc.cpu().numpy()[at]), bits(rk))
        codes, scales = np.zeros((nb, bs, Hkv, D)), np.zeros((nb, 4), np.float32)
        oq.write(rk, qs, tables, lens, codes, scales, bs, "int8")
        assert np.array_equal(codes_of(cache[0], "int8"), codes)


def test_pool_past_32_bits(ops):
    """Blocks whose rows lie past 2^32 elements, and q far along a long batch."""
    rng = np.random.default_rng(2)
    Hq, Hkv, bs = 8, 8, 64
    nb = (1 << 32) // (bs * Hkv * D) + 3
    lens, new = np.array([70, 3], np.int32), [70, 3]
    tables = np.array([[nb - 1, 0], [nb - 2, -1]], np.int32)
    qs, T = starts(new), 73
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    table = table_of(64, 100)
    seq, place = orope.places(qs, lens, T)
    at = tables[seq, place // bs], place % bs
    kc, vc = (torch.zeros((nb, bs, Hkv, D), dtype=torch.float16, device="cuda") for _ in "kv")
    qo = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda")
    err = ops.new_error_word()
    ops.rope_and_cache(qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), kc, vc, dev(table), dev_err=err)
    idx = tuple(dev(a).long() for a in at)
    rk = orope.rotate(k, place, table)
    assert np.array_equal(bits(kc[idx].cpu().numpy()), bits(rk))
    assert np.array_equal(bits(vc[idx].cpu().numpy()), bits(v))
    del kc, vc
    cache = ops.q8_cache(nb, Hkv, bs)
    ops.rope_and_cache_q8(qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), *cache, dev(table), dev_err=err)
    assert ops.read_error_word(err) == 0
    small = np.array([[2, 0], [1, -1]], np.int32)
    codes, scales = np.zeros((3, bs, Hkv, D)), np.zeros((3, 8), np.float32)
    oq.write(rk, qs, small, lens, codes, scales, bs, "int8")
    got = codes_of(cache[0][[0, nb - 2, nb - 1]], "int8")
    assert np.array_equal(got, codes)


@pytest.mark.parametrize("new", [[1, 1, 1], [20, 3, 1]])
def test_q8_tiny_values(ops, new):
    """A table that shrinks keys until their scale has no finite inverse: codes are 0, values are off
    by less than fp32's smallest normal number."""
    rng = np.random.default_rng(5)
    Hq, Hkv, bs = 4, 1, 16
    lens, qs, T = np.array(new, np.int32), starts(new), int(np.sum(new))
    nb, tables = batch(rng, lens, bs)
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    table = (table_of(64, 100) * 1e-38).astype(np.float32)
    cache = ops.q8_cache(nb, Hkv, bs)
    err = ops.new_error_word()
    qo = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda")
    ops.rope_and_cache_q8(qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), *cache, dev(table), dev_err=err)
    assert ops.read_error_word(err) == 0
    seq, place = orope.places(qs, lens, T)
    at = tables[seq, place // bs], place % bs
    got = codes_of(cache[0], "int8")[at] * cache[2].cpu().numpy()[at[0], :Hkv, None]
    ref = orope.rotate(k, place, table)
    off = np.abs(got - ref)
    tiny = np.abs(ref).max(axis=(1, 2)).max() / 127 < 2.0 ** -126
    assert off.max() <= (127 * 2.0 ** -126 if tiny else np.abs(ref).max() / 127)
    codes, scales = np.zeros((nb, bs, Hkv, D)), np.zeros((nb, 4), np.float32)
    oq.write(v, qs, tables, lens, codes, scales, bs, "int8")
    assert np.array_equal(codes_of(cache[1], "int8"), codes)


def test_append_in_place(ops):
    """q_out q itself, a slice of the projection's output, in both caches' calls."""
    rng = np.random.default_rng(6)
    new, Hq, Hkv, bs = [3, 1, 30], 8, 2, 16
    lens, qs, T = np.array(new, np.int32), starts(new), 34
    nb, tables = batch(rng, lens, bs)
    table = table_of(64, 100)
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    _, place = orope.places(qs, lens, T)
    ref = orope.rotate(q, place, table).astype(np.float16)
    kc = torch.zeros((nb, bs, Hkv, D), dtype=torch.float16, device="cuda")
    args = (dev(qs), dev(tables), dev(lens))
    ops.rope_and_cache(tq, tq, tk, tv, *args, kc, torch.zeros_like(kc), dev(table))
    assert np.array_equal(bits(tq.cpu().numpy()), bits(ref))
    assert np.array_equal(bits(tk.cpu().numpy()), bits(k))       # beside it nothing has changed
    ops.rope_and_cache_q8(tq, tq, tk, tv, *args, *ops.q8_cache(nb, Hkv, bs), dev(table))
    assert np.array_equal(bits(tq.cpu().numpy()), bits(orope.rotate(ref, place, table)))
    assert np.array_equal(bits(tv.cpu().numpy()), bits(v))


def test_many_sequences_and_heads(ops):
    """More sequences than a search step holds, more heads than a part does, a long chunk among
    single tokens."""
    rng = np.random.default_rng(7)
    S, Hq, Hkv, bs = 1500, 64, 8, 8
    new = rng.integers(0, 4, S)
    new[700] = 150
    cached = rng.integers(0, 20, S)
    lens, qs, T = (new + cached).astype(np.int32), starts(new), int(new.sum())
    nb, tables = batch(rng, lens, bs)
    table = table_of(64, 400)
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    seq, place = orope.places(qs, lens, T)
    qo = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda")
    cache = ops.q8_cache(nb, Hkv, bs)
    err = ops.new_error_word()
    assert T < 4 * S
    ops.rope_and_cache_q8(qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), *cache, dev(table), dev_err=err)
    assert ops.read_error_word(err) == 0
    at = rng.choice(T, 200, replace=False)
    assert np.array_equal(bits(qo.cpu().numpy()[at]), bits(orope.rotate(q[at], place[at], table)))
    codes = {n: np.zeros((nb, bs, Hkv, D)) for n in "kv"}
    scales = {n: np.zeros((nb, 8), np.float32) for n in "kv"}
    for n, x, c, s in (("k", orope.rotate(k, place, table), cache[0], cache[2]), ("v", v, cache[1], cache[3])):
        oq.write(x, qs, tables, lens, codes[n], scales[n], bs, "int8")
        assert np.array_equal(s.cpu().numpy(), scales[n]) and np.array_equal(codes_of(c, "int8"), codes[n])
    kc = torch.zeros((nb, bs, Hkv, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    ops.rope_and_cache(qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), kc, vc, dev(table), dev_err=err)
    assert ops.read_error_word(err) == 0
    ref = np.zeros((nb, bs, Hkv, D), np.float16)
    ref[tables[seq, place // bs], place % bs] = orope.rotate(k, place, table).astype(np.float16)
    assert np.array_equal(bits(kc.cpu().numpy()), bits(ref))


@pytest.mark.parametrize("adjacent", [0, 1])
def test_positions_of_axes_that_no_pair_follows(ops, native_lib, adjacent):
    """C callers that pass several axes and no axes of the pairs: every pair follows axis 0, and a
    position off the table on any axis leaves its token out, as where the pairs name their axes."""
    rng = np.random.default_rng(8)
    T, Hq, Hkv, bs = 9, 4, 2, 16
    lens, qs = np.array([4, 5], np.int32), starts([4, 5])
    nb, tables = batch(rng, lens, bs)
    (q, k, _), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    table = table_of(64, 50)
    pos = rng.integers(0, 50, (3, T)).astype(np.int32)
    pos[0, 1], pos[1, 4], pos[2, 6] = 50, -1, 50
    gone = np.isin(np.arange(T), [1, 4, 6])
    d = [dev(a) for a in (pos, table, qs, tables, lens)]
    p = [t.data_ptr() for t in d]
    st = torch.cuda.current_stream().cuda_stream
    stride = (Hq + 2 * Hkv) * D

    def run(name):
        qo = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
        ko = torch.full((T, Hkv, D), 7.0, dtype=torch.float16, device="cuda")
        err = ops.new_error_word()
        rot = (p[0], 3, None, p[1], 50, 128, adjacent)
        if name == "rotary":
            rc = native_lib.pkv_rotary_embedding(qo.data_ptr(), ko.data_ptr(), tq.data_ptr(), tk.data_ptr(),
                                                 Hq * D, Hkv * D, stride, stride, *rot, T, Hq, Hkv, D,
                                                 err.data_ptr(), st)
        else:
            cache = ops.q8_cache(nb, Hkv, bs) if name == "q8" else \
                [torch.zeros((nb, bs, Hkv, D), dtype=torch.float16, device="cuda") for _ in "kv"]
            sizes = (T, 2, Hq, Hkv, D, bs, nb, tables.shape[1])
            args = (qo.data_ptr(), tq.data_ptr(), tk.data_ptr(), tv.data_ptr(), Hq * D, stride, stride,
                    stride, p[2], p[3], p[4], *[t.data_ptr() for t in cache])
            if name == "q8":
                rc = native_lib.pkv_rope_and_cache_q8(*args, 0, *rot, *sizes, cache[2].shape[1],
                                                      err.data_ptr(), st)
            else:
                rc = native_lib.pkv_rope_and_cache(*args, *rot, *sizes, err.data_ptr(), st)
        assert rc == 0
        return qo.cpu().numpy(), ko.cpu().numpy(), ops.read_error_word(err)

    for name in ("rotary", "fp16", "q8"):
        qo, ko, err = run(name)
        assert err == 5 and (qo[gone] == 7).all()
        ref = orope.rotate(q[~gone], pos[0, ~gone], table, None, bool(adjacent))
        assert np.array_equal(bits(qo[~gone]), bits(ref))
        if name == "rotary":
            ref = orope.rotate(k[~gone], pos[0, ~gone], table, None, bool(adjacent))
            assert (ko[gone] == 7).all() and np.array_equal(bits(ko[~gone]), bits(ref))


def takes_the_steps_way(new, bs):
    """Which of the 8-bit append's two kernels a batch takes: few tokens a sequence, or long chunks."""
    return sum(new) < max(8, bs // 2) * len(new)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("new,cached", [([100, 64, 40], [3, 60, 0]), ([300], [5]),
                                        ([70, 33, 90, 65], [63, 0, 31, 1])])
def test_q8_long_chunks_not_finite_and_off_the_table(ops, code, bs, new, cached):
    """As test_q8_long_pieces_of_steps, by the kernel of long chunks at every block size: its teams
    exchange their maxima twice for a head whose values are not finite."""
    assert not takes_the_steps_way(new, bs)
    test_q8_long_pieces_of_steps(ops, code, bs, new, cached)


@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("n", [1, 2, 7, 70])
def test_q8_left_out_tokens_start_a_block_of_more_sizes(ops, n, bs):
    test_q8_left_out_tokens_start_a_block(ops, n, bs)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("bs,new", [(64, [40, 1, 1]), (32, [30, 1, 1]), (16, [13, 1, 1, 1]),
                                    (64, [64, 1, 64]), (32, [90, 64])])
@pytest.mark.parametrize("off", ["first", "some", "all"])
def test_q8_pieces_that_begin_with_left_out_tokens(ops, code, bs, new, off):
    """A block that held another sequence's tokens under a large scale: its new rows begin with tokens
    off the table, and the scale comes from the others alone (0 where there are none)."""
    rng = np.random.default_rng([bs, len(new)])
    Hq, Hkv, rows = 5, 3, 100
    lens, qs, T = np.array(new, np.int32), starts(new), sum(new)
    nb, tables = batch(rng, lens, bs)
    (q, k, v), (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    table = table_of(64, rows)
    seq, place = orope.places(qs, lens, T)
    out = {"first": (seq == 0) & (place == 0), "all": seq == 0,
           "some": (seq == 0) & ((place < 3) | (place % 5 == 4))}[off]
    pos = np.where(out, rows, place).astype(np.int32)
    codes = {n: oq.nearest_code(rng.standard_normal((nb, bs, Hkv, D)) * 40, code) for n in "kv"}
    t = {n: codes_to_dev(codes[n], code) for n in "kv"}
    sc = {n: torch.full((nb, 4), 5.0, device="cuda") for n in "kv"}
    qo = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    err = ops.new_error_word()
    ops.rope_and_cache_q8(qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), t["k"], t["v"], sc["k"],
                          sc["v"], dev(table), positions=dev(pos), dev_err=err)
    assert ops.read_error_word(err) == 5
    at = tables[seq, place // bs], place % bs
    for n, x in (("k", orope.rotate(k, place, table)), ("v", v.astype(np.float32))):
        x = x.copy()
        x[out] = 0
        want, scale = codes[n].copy(), np.full((nb, 4), 5.0, np.float32)
        oq.write(x, qs, tables, lens, want, scale, bs, code)
        want[at[0][out], at[1][out]] = codes[n][at[0][out], at[1][out]]    # as they were
        assert np.array_equal(sc[n].cpu().numpy(), scale)
        assert np.array_equal(codes_of(t[n], code), want)
    qo = qo.cpu().numpy()
    assert (qo[out] == 7).all()
    assert np.array_equal(bits(qo[~out]), bits(orope.rotate(q[~out], place[~out], table)))


@pytest.mark.parametrize("new,cached,Hq,Hkv", CASES)
def test_append_equals_two_steps(ops, new, cached, Hq, Hkv):
    """rope_and_cache against rotary_embedding and reshape_and_cache: the same bits of K and V."""
    rng = np.random.default_rng([Hkv, len(new)])
    bs, T = 16, int(np.sum(new))
    lens, qs = (np.array(new) + np.array(cached)).astype(np.int32), starts(new)
    nb, tables = batch(rng, lens, bs)
    _, (tq, tk, tv) = projection(rng, T, Hq, Hkv)
    table = dev(table_of(64, 1000))
    seq, place = orope.places(qs, lens, T)
    one = [torch.zeros((nb, bs, Hkv, D), dtype=torch.float16, device="cuda") for _ in "kv"]
    two = [torch.zeros_like(c) for c in one]
    qo, qo2 = (torch.empty((T, Hq, D), dtype=torch.float16, device="cuda") for _ in range(2))
    ko = torch.empty((T, Hkv, D), dtype=torch.float16, device="cuda")
    ops.rope_and_cache(qo, tq, tk, tv, dev(qs), dev(tables), dev(lens), *one, table)
    ops.rotary_embedding(qo2, ko, tq, tk, dev(place.astype(np.int32)), table)
    slots = tables[seq, place // bs].astype(np.int64) * bs + place % bs
    ops.reshape_and_cache(ko, tv.contiguous(), dev(slots), *two)
    for a, b in zip([qo] + one, [qo2] + two):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
