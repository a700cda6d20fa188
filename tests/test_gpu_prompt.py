"""Prompt attention (packed and over the paged cache) on the GPU against fp64.

Tolerance (derived, elementwise): a softmax weight is rounded to fp16 for the
product with V, at most 2^-11 of itself or, below fp16's normal range, 2^-25 of
the largest weight (at least 1 in the kernel's units).  A score is 128 products
accumulated in fp32, in 8 steps: off by at most 8 * 2^-23 of the sum of their
magnitudes (in log2 units, 1.4427 of that); scaling, the difference to the
maximum and the hardware exp2 add 2^-22 |x| + 2^-21.  The same enters the
denominator.  The product with V is accumulated over n / 16 steps: 2^-23 each.
The result is rounded to fp16 once.
"""
import numpy as np
import pytest
import torch

from oracle import prompt as op
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


def starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def tolerance(ref, spread, peak, mag, vmax, n):
    x = 1.4427 * mag
    rel = 2.0 ** -11 + 2 * (2.0 ** -20 * x + 2.0 ** -22 * x + 2.0 ** -21) + \
        2 * (n / 16 + 16) * 2.0 ** -23
    return (2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 1.01 * rel[:, :, None] * spread +
            n * 2.0 ** -25 * (peak * vmax[None])[:, :, None])


def check(got, q, k, v, first, scale=SCALE):
    ref, spread, peak, mag, vmax = op.attend(q, k, v, first, scale)
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - tolerance(ref, spread, peak, mag, vmax, k.shape[0])
    assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


def run_packed(ops, q, k, v, qs, scale=SCALE, fill=7.0):
    out = torch.full(q.shape, fill, dtype=torch.float16, device="cuda")
    err = ops.new_error_word()
    ops.prompt_attention(out, dev(q), dev(k), dev(v), dev(np.asarray(qs, np.int32)), scale,
                         dev_err=err)
    return out.cpu().numpy(), ops.read_error_word(err)


def paged_case(seed, new, cached, Hq, Hkv, bs, behind=0, poison=True):
    rng = np.random.default_rng(seed)
    lens = (np.array(new) + np.array(cached)).astype(np.int32)
    need = [max(1, wl.blocks_for(int(L), bs)) for L in lens]
    nb = sum(need) + 3
    tables = wl.handout_tables([n * bs for n in need], rng.permutation(nb).astype(np.int32), bs,
                               pad=-9)
    q = wl.host_normal_fp16(rng, (int(np.sum(new)) + behind, Hq, D))
    kc, vc = (wl.host_normal_fp16(rng, (nb, bs, Hkv, D)) for _ in "kv")
    if poison:      # rows that no context holds
        held = np.zeros((nb, bs), bool)
        for s, L in enumerate(lens):
            pos = np.arange(int(L))
            held[tables[s][pos // bs], pos % bs] = True
        kc[~held], vc[~held] = np.nan, np.inf
    return q, kc, vc, tables, lens


def run_paged(ops, q, kc, vc, tables, lens, qs, scale=SCALE, fill=7.0):
    out = torch.full(q.shape, fill, dtype=torch.float16, device="cuda")
    err = ops.new_error_word()
    ops.paged_attention_prefill(out, dev(q), dev(kc), dev(vc), dev(tables), dev(lens),
                                dev(np.asarray(qs, np.int32)), scale, dev_err=err)
    return out.cpu().numpy(), ops.read_error_word(err)


def check_paged(got, q, kc, vc, tables, lens, new, scale=SCALE):
    qs = starts(new)
    for s, n in enumerate(new):
        if n:
            L = int(lens[s])
            check(got[qs[s]:qs[s + 1]], q[qs[s]:qs[s + 1]], op.gather(kc, tables[s], L),
                  op.gather(vc, tables[s], L), L - n, scale)


# ---- packed ------------------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (4, 2), (8, 2), (16, 2), (5, 5)])
@pytest.mark.parametrize("new", [
    [1], [7, 16, 31, 48, 63], [127, 128, 129, 1], [0, 300, 0, 0, 5, 0], [255, 256, 257], [600],
])
def test_packed_matches_oracle(ops, Hq, Hkv, new):
    rng = np.random.default_rng(len(new) * 100 + Hq)
    T = int(np.sum(new))
    q = wl.host_normal_fp16(rng, (T, Hq, D))
    k, v = (wl.host_normal_fp16(rng, (T, Hkv, D)) for _ in "kv")
    qs = starts(new)
    got, err = run_packed(ops, q, k, v, qs)
    assert err == 0
    for s in range(len(new)):
        a, b = qs[s], qs[s + 1]
        if b > a:
            check(got[a:b], q[a:b], k[a:b], v[a:b], 0)


def test_packed_rows_outside_every_sequence(ops):
    """Rows before the first and behind the last sequence: not read (NaN), not written;
    a neighbour's NaN stays with the neighbour."""
    rng = np.random.default_rng(3)
    T = 420
    q = wl.host_normal_fp16(rng, (T, 8, D))
    k, v = (wl.host_normal_fp16(rng, (T, 2, D)) for _ in "kv")
    qs = [9, 150, 290, 401]
    for a in (q, k, v):
        a[:9], a[401:] = np.nan, np.nan
        a[150:290] = np.nan
    got, err = run_packed(ops, q, k, v, qs)
    assert err == 0
    assert (got[:9] == 7).all() and (got[401:] == 7).all()
    for a, b in ((9, 150), (290, 401)):
        check(got[a:b], q[a:b], k[a:b], v[a:b], 0)


def test_first_row_is_its_value(ops):
    """Row 0 of a prompt attends to itself only: its V row, bit for bit."""
    rng = np.random.default_rng(4)
    new = [1, 2, 130]
    q = wl.host_normal_fp16(rng, (133, 4, D))
    k, v = (wl.host_normal_fp16(rng, (133, 4, D)) for _ in "kv")
    got, _ = run_packed(ops, q, k, v, starts(new))
    for a in starts(new)[:-1]:
        assert np.array_equal(got[a], v[a])


@pytest.mark.parametrize("scale", [0.0, -SCALE, 0.7, 1e-4])
def test_scales(ops, scale):
    rng = np.random.default_rng(5)
    q = wl.host_normal_fp16(rng, (300, 4, D))
    k, v = (wl.host_normal_fp16(rng, (300, 2, D)) for _ in "kv")
    got, err = run_packed(ops, q, k, v, [0, 300], scale)
    assert err == 0
    check(got, q, k, v, 0, scale)


@pytest.mark.parametrize("kind", ["climb", "fall", "saw", "late", "masked"])
def test_softmax_bookkeeping(ops, kind):
    """Scores that climb or fall through the prompt by hundreds of log2 units, so that the
    maximum moves in most tiles; a dominant last key; dominant keys that are masked
    for the rows before them."""
    rng = np.random.default_rng(6)
    n = 700
    q = np.zeros((n, 4, D), np.float16)
    q[..., 0] = 8
    q[..., 1:] = rng.standard_normal((n, 4, D - 1)) * 0.3
    k = (rng.standard_normal((n, 2, D)) * 0.3).astype(np.float16)
    v = wl.host_normal_fp16(rng, (n, 2, D))
    t = np.arange(n)
    ramp = {"climb": t / 2, "fall": -t / 2, "saw": (t % 90) * 3.0, "late": np.where(t == n - 1, 400, 0),
            "masked": np.where(t % 128 == 127, 400.0, 0)}[kind]
    k[..., 0] = ramp[:, None]
    got, err = run_packed(ops, q, k, v, [0, n])
    assert err == 0
    check(got, q, k, v, 0)


# ---- over the paged cache ---------------------------------------------------------------

@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (4, 2), (8, 2), (16, 2), (3, 3)])
@pytest.mark.parametrize("new,cached", [
    ([1, 1, 1], [0, 15, 300]),
    ([7, 16, 31, 0, 63], [0, 1, 64, 33, 129]),
    ([130, 257], [700, 3]),
    ([5, 300], [1100, 0]),
])
def test_paged_matches_oracle(ops, bs, Hq, Hkv, new, cached):
    q, kc, vc, tables, lens = paged_case(bs + Hq, new, cached, Hq, Hkv, bs, behind=4)
    got, err = run_paged(ops, q, kc, vc, tables, lens, starts(new))
    assert err == 0
    check_paged(got, q, kc, vc, tables, lens, new)
    assert (got[int(np.sum(new)):] == 7).all()      # rows behind the last sequence


@pytest.mark.parametrize("new,cached", [([3], [5000]), ([8, 1, 2], [4090, 9000, 100]),
                                        ([140, 1], [2500, 0])])
def test_paged_split_keys(ops, new, cached):
    """Few rows over long contexts: the key axis is split and merged."""
    q, kc, vc, tables, lens = paged_case(11, new, cached, 8, 2, 16)
    assert ops.prefill_workspace_bytes(q.shape[0], len(new), 8, 2, tables.shape[1]) > 0
    got, err = run_paged(ops, q, kc, vc, tables, lens, starts(new))
    assert err == 0
    check_paged(got, q, kc, vc, tables, lens, new)


@pytest.mark.parametrize("tail", [127, 128, 129, 255, 256, 257, 384, 640, 1000])
def test_paged_rows_in_one_tile(ops, tail):
    """Chunks whose rows fill one query tile or less, over 1 to 8 KV tiles: both halves
    of the kernel work on them, on every other KV tile each."""
    for Hq, Hkv, n in ((2, 2, 100), (8, 1, 16), (8, 1, 3), (4, 1, 1)):
        new, cached = [n, n + 1], [tail - n if tail > n else 0, tail]
        q, kc, vc, tables, lens = paged_case(tail + Hq, new, cached, Hq, Hkv, 16)
        got, err = run_paged(ops, q, kc, vc, tables, lens, starts(new))
        assert err == 0
        check_paged(got, q, kc, vc, tables, lens, new)


@pytest.mark.parametrize("bs", [8, 16, 64])
def test_many_units_of_every_kind(ops, bs):
    """More units than the GPU has SMs, of one tile and of two, one KV tile and many, in
    one launch: each SM goes through several, in the order they come."""
    rng = np.random.default_rng(bs)
    new = rng.choice([0, 1, 5, 31, 64, 65, 127, 128, 200, 256, 300], size=48)
    cached = rng.choice([0, 0, 7, 100, 129, 640], size=48)
    q, kc, vc, tables, lens = paged_case(19, new, cached, 16, 8, bs, behind=9)
    assert ops.prefill_workspace_bytes(q.shape[0], 48, 16, 8, tables.shape[1], bs) == 0
    got, err = run_paged(ops, q, kc, vc, tables, lens, starts(new))
    assert err == 0
    check_paged(got, q, kc, vc, tables, lens, new)
    assert (got[int(new.sum()):] == 7).all()
    again, _ = run_paged(ops, q, kc, vc, tables, lens, starts(new))
    assert np.array_equal(got, again)


def test_paged_split_bookkeeping(ops):
    """Maxima that lie hundreds of log2 units apart between the splits."""
    q, kc, vc, tables, lens = paged_case(12, [6], [6000], 4, 1, 16)
    q[...] = 0
    q[..., 0] = 8
    L = int(lens[0])
    pos = np.arange(L)
    for f in (0.06, -0.06):
        kc[tables[0][pos // 16], pos % 16, 0, 0] = (f * pos).astype(np.float16)
        got, err = run_paged(ops, q, kc, vc, tables, lens, [0, 6])
        assert err == 0
        check_paged(got, q, kc, vc, tables, lens, [6])


def test_same_bits_whatever_the_placement(ops):
    """Block ids and repeats leave the bits alone."""
    new, cached = [200, 33, 129], [100, 0, 500]
    q, kc, vc, tables, lens = paged_case(13, new, cached, 8, 2, 16, poison=False)
    a, _ = run_paged(ops, q, kc, vc, tables, lens, starts(new))
    b, _ = run_paged(ops, q, kc, vc, tables, lens, starts(new))
    assert np.array_equal(a, b)
    perm = np.random.default_rng(0).permutation(kc.shape[0])
    inv = np.argsort(perm)
    moved = np.where(tables >= 0, inv[np.maximum(tables, 0)], tables).astype(np.int32)
    c, _ = run_paged(ops, q, kc[perm], vc[perm], moved, lens, starts(new))
    assert np.array_equal(a, c)


def test_bad_metadata_is_reported_and_left_out(ops):
    new, cached = [40, 50, 60], [10, 20, 30]
    q, kc, vc, tables, lens = paged_case(14, new, cached, 8, 2, 16)
    qs = starts(new)

    def fine(got, which):
        for s in which:
            L = int(lens[s])
            check(got[qs[s]:qs[s + 1]], q[qs[s]:qs[s + 1]], op.gather(kc, tables[s], L),
                  op.gather(vc, tables[s], L), L - new[s])

    for n in (-1, 49, 16 * tables.shape[1] + 1, 2 ** 31 - 1):
        bad = lens.copy()
        bad[1] = n
        got, err = run_paged(ops, q, kc, vc, tables, bad, qs)
        assert err == 2 and (got[40:90] == 7).all()
        fine(got, (0, 2))
    got, err = run_paged(ops, q, kc, vc, tables, lens, [0, 40, 90, 151])
    assert err == 7 and (got[90:] == 7).all()
    fine(got, (0, 1))
    got, err = run_paged(ops, q, kc, vc, tables, lens, [-1, 40, 90, 150])
    assert err == 7 and (got[:40] == 7).all()
    fine(got, (1, 2))
    for bad_id in (-1, kc.shape[0], 2 ** 31 - 1):
        t = tables.copy()
        t[2, 1] = bad_id
        got, err = run_paged(ops, q, kc, vc, t, lens, qs)
        assert err == 1
        fine(got, (0, 1))
        kz, vz = kc.copy(), vc.copy()      # the block counts as zeros
        kz[tables[2, 1]] = vz[tables[2, 1]] = 0
        check(got[90:150], q[90:150], op.gather(kz, tables[2], 90), op.gather(vz, tables[2], 90), 30)


def test_nothing_to_do(ops):
    q = torch.zeros((0, 8, D), dtype=torch.float16, device="cuda")
    k = torch.zeros((0, 2, D), dtype=torch.float16, device="cuda")
    qs = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert ops.prompt_attention(q, q, k, k, qs, SCALE) is q
    got, err = run_packed(ops, np.zeros((3, 8, D), np.float16), np.zeros((3, 2, D), np.float16),
                          np.zeros((3, 2, D), np.float16), [0, 0, 0])
    assert err == 0 and (got == 7).all()


def test_many_sequences(ops):
    """2,000 prompts of 0 .. 3 tokens: every sequence is found."""
    rng = np.random.default_rng(15)
    new = rng.integers(0, 4, size=2000)
    T = int(new.sum())
    q, k, v = (wl.host_normal_fp16(rng, (T, 1, D)) for _ in "qkv")
    qs = starts(new)
    got, err = run_packed(ops, q, k, v, qs)
    assert err == 0
    for s in range(2000):
        a, b = qs[s], qs[s + 1]
        if b > a:
            check(got[a:b], q[a:b], k[a:b], v[a:b], 0)


def test_graph_and_streams(ops):
    new, cached = [40, 130], [900, 60]
    q, kc, vc, tables, lens = paged_case(16, new, cached, 8, 2, 16)
    args = [dev(a) for a in (q, kc, vc, tables, lens, starts(new))]
    out, out2 = torch.zeros_like(args[0]), torch.zeros_like(args[0])
    n = ops.prefill_workspace_bytes(q.shape[0], 2, 8, 2, tables.shape[1])
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.paged_attention_prefill(out, *args, SCALE, workspace=ws)
    rng = np.random.default_rng(17)
    q = wl.host_normal_fp16(rng, q.shape)
    args[0].copy_(dev(q))
    g.replay()
    torch.cuda.synchronize()
    check_paged(out.cpu().numpy(), q, kc, vc, tables, lens, new)
    side = torch.cuda.Stream()
    launch = ops.paged_attention_prefill(out2, *args, SCALE, stream=side, prepare=True)
    torch.cuda.synchronize()
    launch()
    launch()
    side.synchronize()
    assert torch.equal(out, out2)


def test_wrappers_refuse(ops):
    q = torch.zeros((4, 8, D), dtype=torch.float16, device="cuda")
    k = torch.zeros((4, 2, D), dtype=torch.float16, device="cuda")
    qs = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    kc = torch.zeros((4, 16, 2, D), dtype=torch.float16, device="cuda")
    t = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    n = torch.full((1,), 4, dtype=torch.int32, device="cuda")
    for bad in (lambda: ops.prompt_attention(q, q.bfloat16(), k, k, qs, 1.0),
                lambda: ops.prompt_attention(q, q, k, k, qs.long(), 1.0),
                lambda: ops.prompt_attention(q, q, k.cpu(), k, qs, 1.0),
                lambda: ops.paged_attention_prefill(q, q, kc.float(), kc, t, n, qs, 1.0)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ops.prompt_attention(q, q, k[:3], k[:3], qs, 1.0),
                lambda: ops.prompt_attention(q[:, ::2], q[:, ::2], k, k, qs, 1.0),
                lambda: ops.prompt_attention(q, q, k, k, qs[:0], 1.0),
                lambda: ops.paged_attention_prefill(q, q, kc, kc, t, n, qs[:1], 1.0),
                lambda: ops.paged_attention_prefill(q, q, kc, kc[:2], t, n, qs, 1.0)):
        with pytest.raises(ValueError):
            bad()
    from paged_kv_cache_138_gb300._lib import PagedKVError
    with pytest.raises(PagedKVError):
        ops.prompt_attention(q[:, :6].contiguous(), q[:, :6].contiguous(), k, k, qs, 1.0)


# ---- infinities and NaN in a context's own V -----------------------------------------------

def check_nonfinite(got, q, k, v, first):
    """Values of V that are not finite reach the rows that see their token, in their
    column, and no others: those match the definition with zeros in their place."""
    bad = ~np.isfinite(v)                                            # [L, Hkv, D]
    n, Hq = q.shape[:2]
    L, Hkv = v.shape[:2]
    see = np.arange(L)[None] <= (first + np.arange(n))[:, None]
    hit = np.einsum("nl,lgd->ngd", see.astype(np.int64), bad.astype(np.int64)) > 0
    hit = np.repeat(hit, Hq // Hkv, axis=1)
    clean = np.where(bad, np.float16(0), v)
    ref, spread, peak, mag, vmax = op.attend(q, k, clean, first, SCALE)
    got = np.asarray(got, np.float64)
    assert np.array_equal(~np.isfinite(got), hit)
    over = np.abs(got - ref) - tolerance(ref, spread, peak, mag, vmax, L)
    assert over[~hit].max(initial=-1) <= 0, over[~hit].max()
    for sign in (1, -1):        # one infinity and nothing else in the column: its sign
        inf = np.where(bad, np.where(v == sign * np.inf, 1, 10 ** 6), 0)
        only = np.repeat(np.einsum("nl,lgd->ngd", see.astype(np.int64), inf), Hq // Hkv, axis=1) == 1
        assert (got[only] == sign * np.inf).all()


def plant(rng, v, tokens):
    for t in tokens:
        g, d = rng.integers(v.shape[1]), rng.choice(D, 3, replace=False)
        v[t, g, d] = [np.inf, -np.inf, np.nan]


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("n", [2, 40, 128, 129, 257, 600])
def test_packed_nonfinite_values_reach_later_rows_only(ops, Hq, Hkv, n):
    rng = np.random.default_rng(n + Hq)
    new = [5, n, 30]
    T = sum(new)
    q = wl.host_normal_fp16(rng, (T, Hq, D))
    k, v = (wl.host_normal_fp16(rng, (T, Hkv, D)) for _ in "kv")
    qs = starts(new)
    plant(rng, v, {int(qs[1]) + t for t in (n - 1, n // 2, min(n - 1, 127), min(n - 1, 130))})
    got, err = run_packed(ops, q, k, v, qs)
    assert err == 0
    for s in range(len(new)):
        a, b = qs[s], qs[s + 1]
        check_nonfinite(got[a:b], q[a:b], k[a:b], v[a:b], 0)


@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("Hq,Hkv,new,cached", [
    (8, 8, [200, 3], [77, 500]),         # several tiles; a pair of warpgroups on one tile's rows
    (8, 2, [70, 129], [0, 127]),
    (8, 1, [9, 1, 2], [1000, 1500, 30]),
    (8, 2, [6, 40], [4000, 2500]),       # a split key axis
])
def test_paged_nonfinite_values_reach_later_rows_only(ops, bs, Hq, Hkv, new, cached):
    rng = np.random.default_rng(bs + sum(new))
    q, kc, vc, tables, lens = paged_case(bs, new, cached, Hq, Hkv, bs)
    for s, n in enumerate(new):
        for t in {int(lens[s]) - 1, int(lens[s]) - 1 - n // 2, max(0, int(lens[s]) - n)}:
            row = vc[tables[s][t // bs], t % bs][None]
            plant(rng, row, [0])
    got, err = run_paged(ops, q, kc, vc, tables, lens, starts(new))
    assert err == 0
    qs = starts(new)
    for s, n in enumerate(new):
        L = int(lens[s])
        check_nonfinite(got[qs[s]:qs[s + 1]], q[qs[s]:qs[s + 1]], op.gather(kc, tables[s], L),
                        op.gather(vc, tables[s], L), L - n)


def test_all_values_nan_but_the_first_rows(ops):
    """Every V row from token 37 on is NaN: rows 0 .. 36 are untouched by it."""
    rng = np.random.default_rng(12)
    n = 300
    q = wl.host_normal_fp16(rng, (n, 4, D))
    k, v = (wl.host_normal_fp16(rng, (n, 4, D)) for _ in "kv")
    v[37:] = np.nan
    got, err = run_packed(ops, q, k, v, [0, n])
    assert err == 0
    check_nonfinite(got, q, k, v, 0)


def test_scale_that_is_nan(ops):
    """A NaN for a scale gives NaN, not the result of some other scale."""
    rng = np.random.default_rng(13)
    q, k, v = (wl.host_normal_fp16(rng, (140, 2, D)) for _ in "qkv")
    got, err = run_packed(ops, q, k, v, [0, 140], float("nan"))
    assert err == 0 and np.isnan(got).all()
