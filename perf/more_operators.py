"""What is measured of the rotary-position operators and of 8-bit chunk attention.

Four operators that follow a model's projections, each in a plain form
(elementary torch operations in 32 bits, rounded once at the end) and as the call
a user makes:

  rotary      q and k rotated by their positions, on one axis or on three
  append      the same, and k and v written to the paged fp16 cache
  append_q8   the same into an 8-bit cache (int8 or e4m3 codes, one fp32 scale
              for each block and KV head)
  chunk_q8    causal attention of packed new tokens over the 8-bit cache

q, k and v are slices of one projection's output [T, (heads + 2 kv_heads) 128], as a
model has them.  All shapes have head_dim 128.  Lengths and positions come from
the case alone (`lens_seed`), values from the seed given to `prepare`.
"""
import math

import numpy as np
import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
THETA = 10000.0
QMAX = {"int8": 127.0, "e4m3": 448.0}
#: pairs of each axis for a rotated part of 2 n dims
SECTIONS = {64: (16, 24, 24), 48: (16, 16, 16), 32: (8, 12, 12)}


def _case(name, op, seqs, heads, kv_heads, new, cached=(0, 0), block=16, code="fp16", rot=128,
          axes=1, adjacent=False, lens_seed=1):
    """new / cached: (least, most) tokens of a sequence this call brings / finds in the cache.
    rot: rotated dims of a head; axes: 1 or 3; adjacent: pairs (2j, 2j + 1), else (j, j + rot/2)."""
    return {"name": name, "op": op, "seqs": seqs, "heads": heads, "kv_heads": kv_heads,
            "new_min": new[0], "new_max": new[1], "cached_min": cached[0],
            "cached_max": cached[1], "block": block, "code": code, "rot": rot, "axes": axes,
            "adjacent": adjacent, "lens_seed": lens_seed}


def listed():
    return [
        # one decode step of a 32-head layer: latency
        _case("rotary_step", "rotary", 64, 32, 32, (1, 1), (0, 4095)),
        # prompts with images, positions on three axes
        _case("rotary_images", "rotary", 4, 32, 8, (4096, 4096), axes=3),
        # the smallest decode batch: launch latency
        _case("append_tiny", "append", 5, 8, 8, (1, 1), (6, 62)),
        # one decode step's new tokens of a 40-head layer
        _case("append_step", "append", 64, 40, 40, (1, 1), (0, 4095)),
        # the prompts of a batch of admitted requests
        _case("append_prompts", "append", 16, 32, 8, (1, 4096), (0, 40)),
        # one decode step over an 8-bit cache
        _case("append_q8_step", "append_q8", 256, 32, 8, (1, 1), (0, 4095), code="int8"),
        # the prompts of a batch of admitted requests, half the head rotated, adjacent pairs
        _case("append_q8_prompts", "append_q8", 16, 32, 8, (1, 4096), (0, 40), code="e4m3",
              rot=64, adjacent=True),
        # prompts with images into an 8-bit cache of longer blocks
        _case("append_q8_images", "append_q8", 4, 32, 32, (100, 2500), (0, 600), block=32,
              code="int8", axes=3),
        # the smallest prompts: five requests of 7..63 tokens, launch latency
        _case("chunk_q8_tiny", "chunk_q8", 5, 8, 8, (7, 63), code="int8"),
        # one long prompt of a grouped-head model
        _case("chunk_q8_16k", "chunk_q8", 1, 32, 8, (16384, 16384), code="int8"),
        # prompts whose 2048-token system prefix is already in the cache
        _case("chunk_q8_cached_prefix", "chunk_q8", 8, 32, 32, (64, 512), (2048, 2048),
              code="e4m3"),
        # a few draft tokens checked against long contexts
        _case("chunk_q8_few_rows", "chunk_q8", 4, 32, 8, (5, 8), (30000, 32760), code="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "append_q8", "append_q8", "chunk_q8", "chunk_q8"])
    heads, kv = rng.choice([(8, 8), (32, 32), (40, 40), (32, 8), (16, 8), (64, 8), (8, 1)])
    block = rng.choice([8, 16, 16, 32, 64])
    code = rng.choice(["int8", "e4m3"]) if op.endswith("q8") else "fp16"
    rot, axes, adjacent = rng.choice([128, 128, 96, 64]), rng.choice([1, 1, 3]), rng.random() < 0.4
    lens_seed = rng.randrange(1 << 30)
    if op == "chunk_q8":
        rot, axes, adjacent = 128, 1, False
        seqs = _log(rng, 1, 32)
        cached = rng.choice([0, 0, 700, 2048, 16000])
        most = _log(rng, 1, 16384)
        # no more work than the largest listed prompt
        while seqs * most * (most + 2 * cached) * heads > 16384 * 16384 * 32 and most > 1:
            most = most * 2 // 3
        c = _case("", op, seqs, heads, kv, (max(1, most // 8), max(1, most)), (0, cached), block,
                  code, lens_seed=lens_seed)
    else:
        seqs = _log(rng, 1, 256)
        most = _log(rng, 1, max(2, 54000 * 48 // (seqs * (heads + 2 * kv))))
        c = _case("", op, seqs, heads, kv, (1, most), (0, rng.choice([0, 20, 2000])), block, code,
                  rot, axes, adjacent, lens_seed)
    del c["name"]
    return c


def _lens(case):
    """(new, cached) tokens of each sequence, from the case alone."""
    r = np.random.default_rng([case["lens_seed"], case["seqs"]])
    new = r.integers(case["new_min"], case["new_max"], size=case["seqs"], endpoint=True)
    cached = r.integers(case["cached_min"], case["cached_max"], size=case["seqs"], endpoint=True)
    return new.astype(np.int64), cached.astype(np.int64)


def _places(case):
    """(sequence, place in it) of every packed row."""
    new, cached = _lens(case)
    seq = np.repeat(np.arange(case["seqs"]), new)
    return seq, np.arange(new.sum()) - np.repeat(np.cumsum(new) - new, new) + cached[seq]


def _positions(case):
    """int [axes, T].  Three axes: 32 tokens of text, then an image of 24 x 24, and so on."""
    at = _places(case)[1]
    if case["axes"] == 1:
        return at[None]
    k, r = at // (32 + 576), at % (32 + 576)
    p = np.maximum(r - 32, 0)
    base = k * 56 + np.minimum(r, 32)
    return np.stack([base, base + p // 24, base + p % 24])


def _axes(case):
    """The axis of every pair."""
    n = case["rot"] // 2
    return (0,) * n if case["axes"] == 1 else sum(((a,) * m for a, m in enumerate(SECTIONS[n])), ())


def work(case):
    new, cached = _lens(case)
    ctx = new + cached
    T, total = int(new.sum()), int(ctx.sum())
    Hq, Hkv, bs = case["heads"], case["kv_heads"], case["block"]
    if case["op"] == "chunk_q8":
        blocks = int((-(-ctx // bs)).sum())
        pairs = float((new * cached + new * (new + 1) // 2).sum())
        return {"bytes": 2 * T * Hq * D * 2 + 2 * total * Hkv * D + 2 * blocks * Hkv * 4,
                "flops": 4.0 * D * Hq * pairs}
    axes = np.array(_axes(case))
    rows = sum(np.unique(p).size * int((axes == a).sum()) for a, p in enumerate(_positions(case)))
    b = 2 * T * Hq * D * 2 + 8 * rows + 2 * T * Hkv * D * 2
    if case["op"] == "append":
        b += 2 * T * Hkv * D * 2
    if case["op"] == "append_q8":
        touched = int((-(-ctx // bs) - cached // bs).sum())
        b += 2 * T * Hkv * D + 2 * touched * Hkv * 4
    return {"bytes": b, "flops": 3.0 * T * (Hq + Hkv) * case["rot"]}


# ---- the 8-bit code ----------------------------------------------------------------
# A block's rows of one KV head share one fp32 scale, amax / QMAX; a code stands
# for code * scale.  Codes are those nearest to x * (1 / scale), ties to even.

def _scale_of(amax, code):
    # a tensor divisor: torch multiplies by the inverse of a plain number instead
    return amax / torch.full((), QMAX[code], device=amax.device)


def _inverse(scale):
    return torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))


def _codes(y, code):
    if code == "int8":
        return torch.round(y).clamp(-127, 127).to(torch.int8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 131 + 7)
    # some channels of keys are several times larger than the others
    loud = torch.ones(D, device="cuda")
    loud[torch.randint(0, D, (4,), generator=g, device="cuda")] = 6.0
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda").half()  # noqa: E731
    new, cached = _lens(case)
    S, T, bs, Hkv, Hq = case["seqs"], int(new.sum()), case["block"], case["kv_heads"], case["heads"]
    op, ctx = case["op"], new + cached
    start = np.concatenate([[0], np.cumsum(new)])
    st = {"op": op, "code": case["code"], "block": bs, "start": start.tolist(), "ctx": ctx.tolist()}
    st["q_out"] = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda")
    if op == "chunk_q8":
        st["q"] = normal(T, Hq, D)
    else:
        qkv = normal(T, Hq + 2 * Hkv, D)
        qkv[:, Hq:Hq + Hkv] *= loud.half()
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = _positions(case)
        st["axes"] = _axes(case) if case["axes"] > 1 else None
        st["adjacent"], st["rot"] = case["adjacent"], case["rot"]
        # the program's table of cosines and sines, angles in 64 bits
        n = case["rot"] // 2
        angle = torch.arange(int(pos.max()) + 1, device="cuda").double()[:, None] * \
            THETA ** (-torch.arange(n, device="cuda").double() / n)
        st["table"] = torch.stack([angle.cos(), angle.sin()], dim=-1).float()
        # a cache's positions follow from its lengths where there is one axis
        st["positions"] = torch.from_numpy(pos.astype(np.int32)).cuda() \
            if op == "rotary" or case["axes"] > 1 else None
    if op == "rotary":
        st["k_out"] = torch.empty((T, Hkv, D), dtype=torch.float16, device="cuda")
        return st
    st["query_start"] = torch.from_numpy(start.astype(np.int32)).cuda()
    st["context_lens"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
    # blocks scattered over a pool a tenth larger than what is needed
    need = -(-ctx // bs)
    nb = int(math.ceil(1.1 * need.sum()))
    order = np.random.default_rng(int(seed) * 31 + 5).permutation(nb).astype(np.int32)
    tables = np.full((S, int(need.max())), -1, np.int32)
    ends = np.cumsum(need)
    for s in range(S):
        tables[s, :need[s]] = order[ends[s] - need[s]:ends[s]]
    st["tables"] = torch.from_numpy(tables).cuda()
    if op == "append":
        st["k_cache"], st["v_cache"] = normal(nb, bs, Hkv, D), normal(nb, bs, Hkv, D)
        return st
    # the 8-bit cache as earlier writes left it: rows before this call's tokens
    # hold codes under their block's scale, rows past them hold nothing
    held = np.zeros(nb, np.int64)
    for s in range(S):
        keep = int(ctx[s]) if op == "chunk_q8" else int(cached[s])
        b = tables[s, :-(-keep // bs)] if keep else tables[s, :0]
        held[b] = bs
        if keep % bs:
            held[b[-1]] = keep % bs
    valid = (torch.arange(bs, device="cuda")[None] < torch.from_numpy(held).cuda()[:, None])
    pad = -(-Hkv // 4) * 4
    for n in "kv":
        x = normal(nb, bs, Hkv, D).float() * valid[:, :, None, None]
        if n == "k":
            x *= loud
        scale = _scale_of(x.abs().amax(dim=(1, 3)), case["code"])
        st[n + "_cache"] = _codes(x * _inverse(scale)[:, None, :, None], case["code"])
        st[n + "_scale"] = torch.zeros((nb, pad), device="cuda")
        st[n + "_scale"][:, :Hkv] = scale
        del x
    return st


# ---- the plain forms ----------------------------------------------------------------

def _turn(st):
    """cos and sin [T, 1, n] of every row's pairs."""
    n = st["rot"] // 2
    if st.get("positions") is not None:
        pos = st["positions"].long()
    else:
        pos = _where(st)[2][None]
    axis = torch.tensor(st["axes"] or (0,) * n, device=pos.device)
    at = st["table"][pos[axis].T, torch.arange(n, device=pos.device)]
    return at[:, None, :, 0], at[:, None, :, 1]


def _rotated(x, cos, sin, st):
    """x [T, H, D] rotated, 32 bits."""
    x, rot = x.float(), st["rot"]
    if st["adjacent"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1 if st["adjacent"] else -2)
    return torch.cat([y.flatten(-2), x[..., rot:]], dim=-1)


def _where(st):
    """(block, row in it, place in its sequence) of every packed row."""
    qs, bs = st["query_start"].long(), st["block"]
    i = torch.arange(st["q"].shape[0], device=qs.device)
    s = torch.searchsorted(qs, i, right=True) - 1
    pos = st["context_lens"].long()[s] - (qs[s + 1] - i)
    return st["tables"].long()[s, pos // bs], pos % bs, pos


def _plain_rotary(st):
    turn = _turn(st)
    return [_rotated(st[n], *turn, st).half() for n in "qk"]


def _plain_append(st):
    turn = _turn(st)
    blk, row, _ = _where(st)
    st["k_cache"][blk, row] = _rotated(st["k"], *turn, st).half()
    st["v_cache"][blk, row] = st["v"]
    return [_rotated(st["q"], *turn, st).half(), st["k_cache"], st["v_cache"]]


def _code_rows(x, cache, scales, blk, row, touched, unit, code):
    """New rows x (32 bits) at (blk, row); unit: index of blk among `touched`."""
    Hkv = x.shape[1]
    amax = torch.zeros((touched.numel(), Hkv), device=x.device).index_reduce_(
        0, unit, x.abs().amax(dim=2), "amax")
    first = torch.full((touched.numel(),), 1 << 30, dtype=torch.int64, device=x.device)
    first.scatter_reduce_(0, unit, row, "amin")
    before = torch.where(first[:, None] > 0, scales[touched, :Hkv], torch.zeros_like(amax))
    scale = torch.maximum(before, _scale_of(amax, code))
    # rows written earlier are coded anew where their block's scale grows
    held = cache[touched].float()
    ratio = torch.where(scale > 0, before / scale, torch.zeros_like(scale))
    again = _codes(held * ratio[:, None, :, None], code)
    grows = (scale > before) & (first[:, None] > 0)
    which = (torch.arange(cache.shape[1], device=x.device)[None, :, None] <
             first[:, None, None]) & grows[:, None, :]
    cache[touched] = torch.where(which[..., None], again.view(torch.int8),
                                 cache[touched].view(torch.int8)).view(cache.dtype)
    cache.view(torch.int8)[blk, row] = _codes(x * _inverse(scale)[unit][:, :, None],
                                              code).view(torch.int8)
    scales[touched, :Hkv] = scale


def _plain_append_q8(st):
    turn = _turn(st)
    blk, row, _ = _where(st)
    touched, unit = torch.unique(blk, return_inverse=True)
    _code_rows(_rotated(st["k"], *turn, st), st["k_cache"], st["k_scale"], blk, row, touched, unit,
               st["code"])
    _code_rows(st["v"].float(), st["v_cache"], st["v_scale"], blk, row, touched, unit, st["code"])
    return [_rotated(st["q"], *turn, st).half(), st["k_cache"], st["v_cache"], st["k_scale"],
            st["v_scale"]]


def _attend(q, k, v, first):
    """softmax(SCALE q k^T) v of one sequence: q [n, Hq, D] at places first ..
    first + n - 1, k and v [L, Hkv, D] in 32 bits, rounded once."""
    n, Hq, _ = q.shape
    L, Hkv, _ = k.shape
    qh = q.float().reshape(n, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
    s = (qh @ k.permute(1, 2, 0)).mul_(SCALE).view(Hkv, Hq // Hkv, n, L)
    pos = torch.arange(first, first + n, device=q.device)
    s.masked_fill_(torch.arange(L, device=q.device)[None] > pos[:, None], -math.inf)
    s = s.sub_(s.amax(dim=-1, keepdim=True)).exp_()
    s = s.div_(s.sum(dim=-1, keepdim=True)).view(Hkv, -1, L)
    o = (s @ v.permute(1, 0, 2)).view(Hkv, Hq // Hkv, n, D)
    return o.permute(2, 0, 1, 3).reshape(n, Hq, D).to(q.dtype)


def _rows(st, n, s):
    """The first ctx[s] tokens of sequence s, in 32 bits."""
    L, bs = st["ctx"][s], st["block"]
    at = st["tables"][s][:-(-L // bs)].long()
    cache = st[n + "_cache"]
    x = cache[at].float() * st[n + "_scale"][at, :cache.shape[2]][:, None, :, None]
    return x.flatten(0, 1)[:L]


def _plain_chunk_q8(st):
    a, ctx = st["start"], st["ctx"]
    return torch.cat([_attend(st["q"][a[s]:a[s + 1]], _rows(st, "k", s), _rows(st, "v", s),
                              ctx[s] - (a[s + 1] - a[s])) for s in range(len(ctx))])


_PLAIN = {"rotary": _plain_rotary, "append": _plain_append, "append_q8": _plain_append_q8,
          "chunk_q8": _plain_chunk_q8}


# ---- the framework's calls -------------------------------------------------------------

def _own(st):
    from paged_kv_cache_138_gb300 import ops
    if st["op"] == "rotary":
        ops.rotary_embedding(st["q_out"], st["k_out"], st["q"], st["k"], st["positions"],
                             st["table"], axes=st["axes"], adjacent=st["adjacent"])
        return [st["q_out"], st["k_out"]]
    if st["op"] == "append":
        ops.rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["query_start"],
                           st["tables"], st["context_lens"], st["k_cache"], st["v_cache"],
                           st["table"], positions=st["positions"], axes=st["axes"],
                           adjacent=st["adjacent"])
        return [st["q_out"], st["k_cache"], st["v_cache"]]
    if st["op"] == "append_q8":
        ops.rope_and_cache_q8(st["q_out"], st["q"], st["k"], st["v"], st["query_start"],
                              st["tables"], st["context_lens"], st["k_cache"], st["v_cache"],
                              st["k_scale"], st["v_scale"], st["table"],
                              positions=st["positions"], axes=st["axes"],
                              adjacent=st["adjacent"])
        return [st["q_out"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]]
    return ops.paged_attention_prefill_q8(st["q_out"], st["q"], st["k_cache"], st["v_cache"],
                                          st["k_scale"], st["v_scale"], st["tables"],
                                          st["context_lens"], st["query_start"], SCALE)


def run(state):
    """append and append_q8 return the cache itself; int8 codes have to be equal."""
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ---- the definitions in 64 bits -------------------------------------------------------

def _exact_turned(st, case):
    """q and k rotated in 64 bits (numpy), the table's numbers taken as they are."""
    table, axes = st["table"].cpu().numpy().astype(np.float64), np.array(_axes(case))
    j = np.arange(len(axes))
    i, k = (2 * j, 2 * j + 1) if case["adjacent"] else (j, j + len(axes))
    turn = table[_positions(case)[axes].T, j][:, None]
    out = []
    for n in "qk":
        x = st[n].cpu().numpy().astype(np.float64)
        a, b = x[..., i], x[..., k]
        x[..., i] = a * turn[..., 0] - b * turn[..., 1]
        x[..., k] = a * turn[..., 1] + b * turn[..., 0]
        out.append(x)
    return out


def _exact_code(y, code):
    """The code nearest to y (numpy, 64 bits), ties to even."""
    if code == "int8":
        return np.clip(np.rint(y), -127, 127)
    y = np.clip(y, -448, 448)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 1e-30))), -6) - 3)
    return np.rint(y / step) * step


def _exact_append(st, case, x, n):
    """The cache (and its scales) with rows x [T, Hkv, D], in 64 bits, appended."""
    code, bs, Hkv = case["code"], case["block"], case["kv_heads"]
    tables = st["tables"].cpu().numpy()
    cache = st[n + "_cache"].float().cpu().numpy().astype(np.float64)
    seq, pos = _places(case)
    if case["op"] == "append":
        cache[tables[seq, pos // bs], pos % bs] = x
        return cache, None
    scale = st[n + "_scale"].cpu().numpy().astype(np.float64)
    # one block of one sequence after another
    cut = np.flatnonzero(np.diff(seq * (1 << 40) + pos // bs, prepend=-1))
    for lo, hi in zip(cut, [*cut[1:], len(seq)]):
        b, r = int(tables[seq[lo], pos[lo] // bs]), int(pos[lo] % bs)
        rows = x[lo:hi]
        old = scale[b, :Hkv].copy() if r else np.zeros(Hkv)
        now = np.maximum(old, np.abs(rows).max(axis=(0, 2)) / QMAX[code])
        grown = now > old
        if r and grown.any():
            y = cache[b, :r][:, grown] * (old[grown] / now[grown])[None, :, None]
            cache[b, :r, grown] = _exact_code(y, code).transpose(1, 0, 2)
        inv = np.divide(1.0, now, out=np.zeros_like(now), where=now > 0)
        cache[b, r:r + hi - lo] = _exact_code(rows * inv[None, :, None], code)
        scale[b, :Hkv] = now
    return cache, scale


def _exact_chunk(st, case):
    Hq, Hkv, bs = case["heads"], case["kv_heads"], case["block"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s in range(case["seqs"]):
        lo, hi, L = st["start"][s], st["start"][s + 1], st["ctx"][s]
        tok = torch.arange(L, device="cuda")
        b = st["tables"][s].long()[tok // bs]
        kv = [st[n + "_cache"][b, tok % bs].double() * st[n + "_scale"][b, :Hkv].double()[:, :, None]
              for n in "kv"]
        for h in range(Hq):
            k, v = (x[:, h * Hkv // Hq] for x in kv)
            for i in range(lo, hi, 2048):
                j = min(hi, i + 2048)
                last = L - hi + j
                w = torch.mm(st["q"][i:j, h].double(), k[:last].T) / math.sqrt(D)
                seen = (L - hi + torch.arange(i, j, device="cuda"))[:, None] >= tok[None, :last]
                w = torch.where(seen, w, torch.full_like(w, -math.inf))
                out[i:j, h] = torch.mm(torch.softmax(w, dim=1), v[:last])
    return out


def exact(case, seed):
    w = work(case)
    if w["flops"] > 2.5e12 if case["op"] == "chunk_q8" else w["bytes"] > 8e8:
        return None
    st = prepare(case, seed)
    if case["op"] == "chunk_q8":
        return _exact_chunk(st, case)
    q, k = _exact_turned(st, case)
    if case["op"] == "rotary":
        return [torch.from_numpy(q), torch.from_numpy(k)]
    v = st["v"].cpu().numpy().astype(np.float64)
    both = [_exact_append(st, case, x, n) for x, n in ((k, "k"), (v, "v"))]
    parts = [q, both[0][0], both[1][0]]
    if case["op"] == "append_q8":
        parts += [both[0][1], both[1][1]]
    return [torch.from_numpy(x) for x in parts]
