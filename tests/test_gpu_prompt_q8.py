"""Prompt attention over the 8-bit cache on the GPU against fp64 over the codes' values.

Tolerance (derived, elementwise): a softmax weight, V scale included, is rounded to fp16 for
the product with V, at most 2^-11 of itself or, below fp16's normal range, 2^-25 of the kernel's
unit, the largest weight being 2^7 units or more: 2^-32 of it for each token, times a code of at
most 448.  A score is 128 products accumulated in fp32, in 8 steps: off by at most 8 * 2^-23 of
the sum of their magnitudes (in log2 units, 1.4427 of that).  The exponent x + log2 v_scale - m
is formed from two rounded factors, a logarithm (2^-21) and two sums of magnitude at most
x + 80 (V scales lie between 2^-33 and 2^17 here): 2^-22 (x + 80) + 2^-21, and the hardware exp2
adds 2^-21.  The same enters the denominator.  The product with V is accumulated over n / 16
steps: 2^-23 each.  The result is rounded to fp16 once.
"""
import numpy as np
import pytest
import torch

import test_gpu_prompt as tp
import test_gpu_q8 as tq
from oracle import q8 as oq
from oracle import rope as orope
from paged_kv_cache_138_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
D = 128
SCALE = 1.0 / np.sqrt(D)
CODES = ["int8", "e4m3"]


@pytest.fixture(scope="module")
def ops(native_lib):
    from paged_kv_cache_138_gb300 import ops as o
    return o


dev, starts = tp.dev, tp.starts


def tolerance(ref, spread, peak, mag, n):
    x = 1.4427 * mag
    rel = 2.0 ** -11 + 2 * (2.0 ** -20 * x + 2.0 ** -22 * (x + 80) + 2.0 ** -20) + \
        2 * (n / 16 + 16) * 2.0 ** -23
    return (2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 1.01 * rel[:, :, None] * spread +
            n * 2.0 ** -32 * 448 * peak[:, :, None])


class Case:
    """A batch over a cache of random codes; rows and blocks that no context holds are poisoned."""

    def __init__(self, seed, new, cached, Hq, Hkv, bs, code, behind=0, width=0, scales=None):
        rng = np.random.default_rng(seed)
        self.code, self.bs, self.new = code, bs, new
        self.lens = (np.array(new) + np.array(cached)).astype(np.int32)
        need = [max(1, wl.blocks_for(int(L), bs)) for L in self.lens]
        self.nb = nb = sum(need) + 3
        self.tables = wl.handout_tables([n * bs for n in need], rng.permutation(nb).astype(np.int32),
                                        bs, pad=-9)
        if width:
            wide = np.full((len(new), width), -9, np.int32)
            wide[:, :self.tables.shape[1]] = self.tables
            self.tables = wide
        self.qs = starts(new)
        self.q = wl.host_normal_fp16(rng, (int(np.sum(new)) + behind, Hq, D))
        self.stride = -(-Hkv // 4) * 4
        self.codes = [oq.nearest_code(rng.standard_normal((nb, bs, Hkv, D)) * 40, code) for _ in "kv"]
        draw = scales or (lambda r, shape, kind: np.abs(r.standard_normal(shape)) * 0.02 + 0.01)
        self.scales = [draw(rng, (nb, self.stride), n).astype(np.float32) for n in "kv"]
        self.held = np.zeros((nb, bs), bool)
        for s, L in enumerate(self.lens):
            pos = np.arange(int(L))
            self.held[self.tables[s][pos // bs], pos % bs] = True

    def device(self):
        """(k_cache, v_cache, k_scale, v_scale) on the device, poisoned."""
        out = []
        for c in self.codes:
            t = tq.codes_to_dev(c, self.code)
            t.view(torch.uint8)[dev(~self.held)] = 0x7f if self.code == "e4m3" else 0x80
            out.append(t)
        for s in self.scales:
            s = s.copy()
            s[~self.held.any(axis=1)] = np.nan
            out.append(dev(s))
        return out

    def run(self, ops, scale=SCALE, fill=7.0, **a):
        out = torch.full(self.q.shape, fill, dtype=torch.float16, device="cuda")
        err = ops.new_error_word()
        ops.paged_attention_prefill_q8(out, dev(self.q), *self.device(), dev(self.tables),
                                       dev(self.lens), dev(self.qs), scale, dev_err=err, **a)
        return out.cpu().numpy(), ops.read_error_word(err)

    def tokens(self, s):
        """Codes and scales of sequence s token by token."""
        pos = np.arange(int(self.lens[s]))
        at, row = self.tables[s][pos // self.bs], pos % self.bs
        H = self.codes[0].shape[2]
        return [c[at, row] for c in self.codes] + [x[at][:, :H] for x in self.scales]

    def check(self, got, scale=SCALE, seqs=None, rows=None):
        for s in range(len(self.new)) if seqs is None else seqs:
            n, L = self.new[s], int(self.lens[s])
            if not n:
                continue
            a, b = self.qs[s], self.qs[s + 1]
            if rows:
                a = max(a, b - rows)
            kc, vc, ks, vs = self.tokens(s)
            ref, spread, peak, mag = oq.chunk(self.q[a:b], kc, vc, ks, vs, L - (b - a), scale)
            y = np.asarray(got[a:b], np.float64)
            assert np.isfinite(y).all(), s
            over = np.abs(y - ref) - tolerance(ref, spread, peak, mag, L)
            assert over.max() <= 0, (s, over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (4, 2), (8, 2), (16, 2), (5, 5)])
@pytest.mark.parametrize("new,cached", [
    ([1], [0]),
    ([7, 16, 31, 48, 63], [0, 0, 0, 0, 0]),
    ([127, 128, 0, 129, 1], [0, 1, 50, 127, 300]),
    ([3, 40], [700, 129]),
    ([300], [513]),
])
def test_matches_oracle(ops, code, bs, Hq, Hkv, new, cached):
    c = Case([bs, Hq, len(new)], new, cached, Hq, Hkv, bs, code, behind=2)
    got, err = c.run(ops)
    assert err == 0
    c.check(got)
    assert (got[int(np.sum(new)):] == 7).all()        # rows that no sequence owns


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("new,cached,bs", [([5, 8, 1], [5000, 4001, 0], 16), ([1], [9000], 64),
                                           ([33], [3000], 8), ([140], [4500], 32)])
def test_split_key_axis(ops, code, new, cached, bs):
    """Few rows over long contexts: several units share a row, and a merge joins them."""
    c = Case(5, new, cached, 8, 2, bs, code, width=wl.blocks_for(9100, bs))
    assert ops.prefill_q8_workspace_bytes(len(c.q), len(new), 8, 2, c.tables.shape[1], bs) > 0
    got, err = c.run(ops)
    assert err == 0
    c.check(got)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("new,cached,Hq,Hkv,bs", [
    ([6000], [0], 32, 8, 16), ([700, 400], [2048, 3000], 8, 8, 16),
    ([5, 8, 6], [12000, 9000, 8000], 8, 2, 16), ([8] * 40, [1500] * 40, 8, 2, 64),
    ([2] * 40, [1500] * 40, 8, 2, 16), ([4] * 20, [1500] * 20, 8, 2, 8),
])
def test_same_bits_every_time(ops, code, new, cached, Hq, Hkv, bs):
    """Launches of two batches one after another, many times: each batch's rows are the same bits
    every time (nothing depends on which copy lands first), and sampled rows are right."""
    cases = [Case([s, bs], new, cached, Hq, Hkv, bs, code) for s in (40, 41)]
    outs, calls = [], []
    for c in cases:
        out = torch.empty(c.q.shape, dtype=torch.float16, device="cuda")
        calls.append(ops.paged_attention_prefill_q8(out, dev(c.q), *c.device(), dev(c.tables),
                                                    dev(c.lens), dev(c.qs), SCALE, prepare=True))
        outs.append(out)
    first = None
    for _ in range(25):
        for out in outs:
            out.fill_(7)
        for _ in range(2):
            for call in calls:
                call()
        torch.cuda.synchronize()
        now = [out.clone() for out in outs]
        first = first or now
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(now, first))
    for c, out in zip(cases, first):
        c.check(out.cpu().numpy(), rows=2)


def split_tokens(ops, c, Hq, Hkv):
    """Tokens of a split of the case's launch, from the workspace's size."""
    T, S, width = len(c.q), len(c.new), c.tables.shape[1]
    splits = ops.prefill_q8_workspace_bytes(T, S, Hq, Hkv, width, c.bs) // (T * Hq * 130 * 4)
    tiles = -(-width * c.bs // 128)
    assert splits > 1
    return -(-tiles // splits) * 128


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("new,Hq,Hkv", [([4, 2, 3], 8, 2), ([8, 8, 5], 4, 4), ([2, 1, 2], 8, 1),
                                        ([20, 9, 30], 4, 2), ([60, 33, 50], 8, 2)])
def test_rows_on_both_sides_of_a_split(ops, code, new, Hq, Hkv):
    """Contexts that end on a split's first tokens: some of a unit's rows see the split, some do
    not, and some have one split less to join."""
    bs, width = 16, 640
    c = Case(30, new, [0] * 3, Hq, Hkv, bs, code, width=width)
    each = split_tokens(ops, c, Hq, Hkv)
    for d in (0, 1, 2, max(new) - 1, max(new)):
        lens = [each + d, 2 * each + d, 3 * each + d]
        lens = [max(n, min(L, width * bs)) for n, L in zip(new, lens)]
        c = Case(31 + d, new, [L - n for n, L in zip(new, lens)], Hq, Hkv, bs, code, width=width)
        assert split_tokens(ops, c, Hq, Hkv) == each
        got, err = c.run(ops)
        assert err == 0
        c.check(got)


@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 2), (8, 1)])
def test_few_rows_with_a_long_chunk_among_them(ops, Hq, Hkv):
    """The kernel for few rows goes by the average: one sequence that brings many is cut into units."""
    new = [1] * 60 + [77, 0, 2, 0, 1] + [1] * 35
    cached = [0, 5, 130, 700, 33] * 20
    c = Case(13, new, cached, Hq, Hkv, 16, "int8")
    got, err = c.run(ops)
    assert err == 0
    c.check(got)


def test_many_units_of_every_kind(ops):
    """Units of one and of two query tiles, long and short, more than there are SMs, so that CTAs go
    from one kind to another; sampled rows against the oracle."""
    rng = np.random.default_rng(8)
    new = [int(n) for n in rng.integers(1, 700, 60)]
    cached = [int(n) for n in rng.choice([0, 0, 5, 130, 900], 60)]
    c = Case(9, new, cached, 8, 4, 16, "int8")
    got, err = c.run(ops)
    assert err == 0
    c.check(got, rows=3)
    c.check(got, seqs=[0, 17, 59])


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("kind", ["spread", "zeros", "tiny"])
def test_scales(ops, code, kind):
    """Scales that differ by 2^12 between blocks, blocks of scale 0, and scales near the least that
    fp16 values can give."""
    def draw(rng, shape, which):
        if kind == "spread":     # K: scores of a few units; V: up to fp16's range
            return np.exp2(rng.uniform(-12, 0, shape)) * (0.05 if which == "k" else 100)
        if kind == "zeros":
            return np.where(rng.random(shape) < 0.5, 0, 0.02)
        return np.exp2(rng.uniform(-33, -24, shape)) if which == "v" else 0.02 + 0 * rng.random(shape)
    c = Case(11, [130, 40], [200, 700], 8, 2, 16, code, scales=draw)
    c.codes = [np.where((s[:, :2] == 0)[:, None, :, None], 0, x) for x, s in zip(c.codes, c.scales)]
    got, err = c.run(ops)
    assert err == 0
    c.check(got)
    assert kind == "zeros" or np.abs(got.astype(np.float64)).max() > 0


@pytest.mark.parametrize("at", ["first", "middle", "late"])
@pytest.mark.parametrize("loud", ["weight", "scale"])
def test_many_small_weights_beside_a_dominant_one(ops, at, loud):
    """32,768 tokens 25 to 29 log2 units below one whose V is 0 in half of the dims: there the others
    make up the output.  The dominant one stands out by its score, or half by its V scale (its
    values are as large as the others')."""
    n = 32768
    c = Case(1, [8], [n - 8], 1, 1, 16, "int8")
    rng = np.random.default_rng(2)
    top = {"first": 0, "middle": n // 2, "late": n - 16}[at]
    c.q[:] = 0
    c.q[..., 0] = 1
    for a in c.codes:
        a[:] = 0
    c.codes[0][..., 0] = -np.round(rng.uniform(101, 116, c.codes[0].shape[:-1]))
    c.scales[0][:] = 0.25
    c.codes[1][:] = np.round(rng.uniform(64, 96, c.codes[1].shape))
    c.scales[1][:] = 2.0 ** -6
    blk, row = c.tables[0][top // 16], top % 16
    c.codes[0][blk, row, 0, 0] = 0
    c.codes[1][blk, row, 0, ::2] = 0
    if loud == "scale":
        c.scales[1][blk] = 2.0 ** 3        # the block's other tokens too
    got, err = c.run(ops, scale=float(np.log(2)))
    assert err == 0
    c.check(got, scale=float(np.log(2)))


@pytest.mark.parametrize("scale", [-SCALE, 0.0, 1e-9, 0.9])
def test_softmax_scales(ops, scale):
    c = Case(3, [70, 5], [100, 0], 8, 2, 16, "int8")
    got, err = c.run(ops, scale=scale)
    assert err == 0
    c.check(got, scale=scale)


def test_not_finite(ops):
    """A NaN or infinity in a row's q, and a softmax scale that is not finite, give NaN there and
    nowhere else."""
    c = Case(4, [70, 5], [100, 0], 8, 2, 16, "e4m3")
    good, err = c.run(ops)
    c.q[3, 1, 7], c.q[40, 6, 100], c.q[72, 0, 0] = np.nan, np.inf, -np.inf
    got, err = c.run(ops)
    assert err == 0
    bad = np.zeros(got.shape[:2], bool)
    bad[3, 1] = bad[40, 6] = bad[72, 0] = True
    assert np.isnan(got[bad]).all()
    assert np.array_equal(got[~bad].view(np.uint16), good[~bad].view(np.uint16))
    for scale in (np.nan, np.inf):
        assert np.isnan(c.run(ops, scale=scale)[0]).all()


def test_bad_metadata(ops):
    c = Case(6, [40, 130, 3], [0, 100, 20], 8, 2, 16, "int8")
    qs, lens, tables = c.qs.copy(), c.lens.copy(), c.tables.copy()
    c.lens[1] = 20
    got, err = c.run(ops)
    assert err == 2 and (got[40:170] == 7).all()
    c.check(got, seqs=[0, 2])
    c.lens = lens.copy()
    c.lens[2] = c.tables.shape[1] * 16 + 1
    got, err = c.run(ops)
    assert err == 2 and (got[170:] == 7).all()
    c.lens, c.qs = lens.copy(), qs.copy()
    c.qs[3] = 174
    got, err = c.run(ops)
    assert err == 7 and (got[170:] == 7).all()
    c.qs = qs
    # a block out of range counts as zeros
    c.tables[1, 2] = c.nb
    got, err = c.run(ops)
    assert err == 1
    c.tables = tables
    for a in c.codes:
        a[tables[1, 2]] = 0
    c.check(got)


def test_decode_steps_agree(ops):
    """A batch of single tokens: the same rows as paged_attention_decode_q8, each within its own
    tolerance of the oracle."""
    c = Case(7, [1] * 6, [0, 15, 16, 300, 1000, 77], 8, 2, 16, "int8")
    got, err = c.run(ops)
    assert err == 0
    c.check(got)
    out = torch.empty((6, 8, D), dtype=torch.float16, device="cuda")
    ops.paged_attention_decode_q8(out, dev(c.q), *c.device(), dev(c.tables), dev(c.lens), SCALE)
    c.check(out.cpu().numpy())


def test_streams_graphs_and_workspaces(ops):
    """Split launches on another stream than the current one, prepared, and two captured graphs with
    a workspace each, replayed one over the other on two streams."""
    cases = [Case(s, [4, 2], [3000, 900], 8, 2, 16, "int8", width=200) for s in (20, 21)]
    need = ops.prefill_q8_workspace_bytes(6, 2, 8, 2, 200)
    assert need > 0
    runs = []
    for c in cases:
        st = torch.cuda.Stream()
        args = [dev(c.q), *c.device(), dev(c.tables), dev(c.lens), dev(c.qs)]
        out = torch.full(c.q.shape, 7.0, dtype=torch.float16, device="cuda")
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        call = ops.paged_attention_prefill_q8(out, *args, SCALE, workspace=ws, stream=st, prepare=True)
        call()
        st.synchronize()
        first = out.cpu().numpy()
        c.check(first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            call()
        runs.append((c, st, graph, out, first, args))
    for _ in range(3):
        for c, st, graph, out, first, _ in runs:
            with torch.cuda.stream(st):
                out.fill_(7)
                graph.replay()
        torch.cuda.synchronize()
        for c, st, graph, out, first, _ in runs:
            assert np.array_equal(out.cpu().numpy().view(np.uint16), first.view(np.uint16))
    # a workspace that the call makes is memory of the launch stream
    c, st, _, out, first, args = runs[0]
    out.fill_(7)
    torch.cuda.synchronize()
    ops.paged_attention_prefill_q8(out, *args, SCALE, stream=st)
    junk = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy().view(np.uint16), first.view(np.uint16)) and junk is not None


def test_pool_past_32_bits(ops):
    """Blocks whose codes lie past 2^32 bytes."""
    c = Case(12, [70, 3], [60, 0], 8, 8, 64, "int8")
    big = (1 << 32) // (64 * 8 * D) + 8
    small = c.device()
    cache = [torch.zeros((big, 64, 8, D), dtype=torch.int8, device="cuda") for _ in "kv"] + \
        [torch.zeros((big, 8), device="cuda") for _ in "kv"]
    for t, s in zip(cache, small):
        t[big - c.nb:] = s
    out = torch.empty(c.q.shape, dtype=torch.float16, device="cuda")
    err = ops.new_error_word()
    tables = np.where(c.tables >= 0, c.tables + big - c.nb, -1).astype(np.int32)
    ops.paged_attention_prefill_q8(out, dev(c.q), *cache, dev(tables), dev(c.lens), dev(c.qs), SCALE,
                                   dev_err=err)
    assert ops.read_error_word(err) == 0
    c.check(out.cpu().numpy())


@pytest.mark.parametrize("code", CODES)
def test_prompts_in_chunks_then_steps(ops, code):
    """As a server uses them: prompts of one batch in chunks, each rotated into the 8-bit cache and
    attended over it, then steps that append and decode; block tables from the BlockManager."""
    from paged_kv_cache_138_gb300.block_manager import BlockManager
    rng = np.random.default_rng(17)
    Hq, Hkv, bs, nb, mb = 8, 2, 16, 120, 40
    bm = BlockManager(nb, bs, enable_prefix_cache=False)
    prompts = [330, 41, 200]
    for s, n in enumerate(prompts):
        bm.allocate(s, rng.integers(0, 32000, size=n).tolist())
    tables, _ = bm.block_tables([0, 1, 2], max_blocks=mb)
    table = ops.rope_table(10000.0 ** (-np.arange(64) / 64), 1024)
    host_table = table.cpu().numpy()
    cache = ops.q8_cache(nb, Hkv, bs, tq.DTYPE[code])
    c = Case.__new__(Case)
    c.code, c.bs = code, bs
    c.codes = [np.zeros((nb, bs, Hkv, D)) for _ in "kv"]
    c.scales = [np.zeros((nb, 4), np.float32) for _ in "kv"]
    err = ops.new_error_word()
    held = np.zeros(3, int)

    def advance(new, attend):
        nonlocal held, tables
        held = held + np.array(new)
        T, lens, qs = int(np.sum(new)), held.astype(np.int32), starts(new)
        x = rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float16)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        qkv = dev(x)
        qo = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda")
        ops.rope_and_cache_q8(qo, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], dev(qs),
                              dev(tables), dev(lens), *cache, table, dev_err=err)
        out = torch.empty_like(qo)
        attend(out, qo, dev(tables), dev(lens), dev(qs))
        _, place = orope.places(qs, lens, T)
        oq.write(orope.rotate(k, place, host_table), qs, tables, lens, c.codes[0], c.scales[0], bs, code)
        oq.write(v, qs, tables, lens, c.codes[1], c.scales[1], bs, code)
        c.q = orope.rotate(q, place, host_table).astype(np.float16)
        c.tables, c.lens, c.qs, c.new = tables, lens, qs, list(new)
        c.check(out.cpu().numpy())

    chunk = lambda out, q, t, n, s: ops.paged_attention_prefill_q8(   # noqa: E731
        out, q, *cache, t, n, s, SCALE, dev_err=err)
    step = lambda out, q, t, n, s: ops.paged_attention_decode_q8(     # noqa: E731
        out, q, *cache, t, n, SCALE, dev_err=err)
    advance([130, 41, 0], chunk)
    advance([130, 0, 200], chunk)
    advance([70, 0, 0], chunk)
    for i in range(20):
        for s in range(3):
            bm.append_slot(s, i)
        tables, _ = bm.block_tables([0, 1, 2], max_blocks=mb)
        advance([1, 1, 1], step if i % 2 else chunk)
    assert ops.read_error_word(err) == 0
    for t, a in zip(cache, c.codes):
        assert np.array_equal(tq.codes_of(t, code), a)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("new,cached,width", [([3], [125], 0), ([130, 40], [200, 700], 0),
                                              ([2, 5], [3000, 40], 200)])
def test_zero_scales_with_codes_left(ops, code, new, cached, width):
    """Blocks of scale 0 are zeros whatever codes lie in them (a block that begins with left-out
    tokens keeps its last owner's): rows that see no other V are exactly 0, others the definition."""
    largest = {"int8": 127, "e4m3": 448}[code]
    c = Case(60, new, cached, 8, 2, 16, code, width=width)
    c.codes[1][:] = largest
    c.scales[1][:] = 0
    got, err = c.run(ops)
    assert err == 0 and (got == 0).all()
    rng = np.random.default_rng(61)
    c = Case(62, new, cached, 8, 2, 16, code, width=width)
    for k in range(2):
        none = rng.random(c.scales[k].shape) < 0.5
        c.scales[k][none] = 0
        c.codes[k] = np.where(none[:, None, :2, None], -largest, c.codes[k])
    got, err = c.run(ops)
    assert err == 0
    c.check(got)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("new,cached,Hq,Hkv,width", [
    ([200, 3], [77, 500], 4, 4, 0),        # units of two tiles; a pair of warpgroups on one
    ([60, 40], [4000, 2500], 8, 2, 640),   # a split key axis, units of one tile
    ([2, 5], [4000, 2500], 8, 2, 640),     # the kernel for few rows, split
])
def test_scores_that_are_all_minus_infinity(ops, code, new, cached, Hq, Hkv, width):
    """An infinity in q where the keys have the other sign: NaN, as the softmax of such a row is,
    and the rows beside it the same bits as without it."""
    c = Case(63, new, cached, Hq, Hkv, 16, code, width=width)
    c.codes[0][..., 3] = -np.maximum(np.abs(c.codes[0][..., 3]), 1)
    clean, err = c.run(ops)
    assert err == 0 and np.isfinite(clean).all()
    q = c.q
    for i in (0, new[0] - 1, new[0]):
        c.q = q.copy()
        c.q[i, 1, 3] = np.inf
        got, err = c.run(ops)
        want = clean.copy()
        want[i, 1] = np.nan
        assert err == 0 and np.array_equal(got, want, equal_nan=True), i
