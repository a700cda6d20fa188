"""TEST INFRASTRUCTURE ONLY: the 8-bit cache's write and decode attention in NumPy.

Codes are held as the float64 values they stand for before scaling (-127..127,
or the finite e4m3 values).  The write follows the operator's definition, its
quotients and products rounded to fp32; attention is the plain definition in
fp64 over code * scale.
"""
import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0}


def nearest_code(y, code):
    """The code nearest to y (float64), ties to even, saturating."""
    y = np.asarray(y, dtype=np.float64)
    if code == "int8":
        return np.clip(np.rint(y), -127, 127)
    y = np.clip(y, -448, 448)
    # spacing of e4m3 at |y|: 2^(e - 3), e >= -6 (subnormals below 2^-6)
    e = np.frexp(np.where(y == 0, 1.0, y))[1] - 1
    step = np.exp2(np.maximum(e, -6) - 3.0)
    return np.where(y == 0, 0.0, np.rint(y / step) * step)


def e4m3_bits_to_value(b):
    """The value of each e4m3 byte (NaN for 0x7f and 0xff)."""
    b = np.asarray(b, dtype=np.uint8).astype(np.int64)
    sign, e, m = np.where(b & 0x80, -1.0, 1.0), (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    return np.where((b & 0x7f) == 0x7f, np.nan, sign * v)


def write(x, query_start, tables, lens, codes, scales, block_size, code):
    """In place: packed rows x [T, H, D] into codes [nb, bs, H, D] (float64) and scales
    [nb, >= H] (float32)."""
    f32, H = np.float32, x.shape[1]
    x = np.asarray(x, dtype=np.float32)
    x = np.where(np.isfinite(x), x, f32(0))
    for s in range(len(lens)):
        a, b = int(query_start[s]), int(query_start[s + 1])
        pos0 = int(lens[s]) - (b - a)
        blocks = {}
        for i in range(a, b):
            pos = pos0 + i - a
            blocks.setdefault(pos // block_size, []).append((pos % block_size, i))
        for lb, rows in blocks.items():
            blk, first = int(tables[s][lb]), rows[0][0]
            for h in range(H):
                new = x[[i for _, i in rows], h]
                s0 = scales[blk, h] if first > 0 else f32(0)
                s1 = max(s0, f32(np.abs(new).max()) / f32(QMAX[code]))
                if first > 0 and s1 > s0:
                    old = codes[blk, :first, h].astype(f32) * f32(s0 / s1)
                    codes[blk, :first, h] = nearest_code(old, code)
                inv = f32(1) / s1 if s1 > 0 else f32(0)
                for (r, _), v in zip(rows, new):
                    codes[blk, r, h] = nearest_code(v * inv, code)
                scales[blk, h] = s1


def decode(q, k_codes, v_codes, k_scale, v_scale, tables, lens, scale, block_size):
    """(out, slack): fp64 attention over code * scale and, for every output, the sum
    of weight * |V| and the weights' largest share, for error bounds."""
    S, Hq, D = q.shape
    Hkv = k_codes.shape[2]
    out = np.zeros((S, Hq, D))
    spread = np.zeros((S, Hq, D))
    peak = np.zeros((S, Hq))
    top = np.zeros((S, Hq))
    for s in range(S):
        L = int(lens[s])
        if L == 0:
            continue
        pos = np.arange(L)
        blk, row = np.asarray(tables[s])[pos // block_size], pos % block_size
        for h in range(Hq):
            g = h // (Hq // Hkv)
            ks, vs = k_scale[blk, g].astype(np.float64), v_scale[blk, g].astype(np.float64)
            x = scale * (k_codes[blk, row, g] @ q[s, h].astype(np.float64)) * ks
            p = np.exp(x - x.max())
            p /= p.sum()
            v = v_codes[blk, row, g] * vs[:, None]
            out[s, h] = p @ v
            spread[s, h] = p @ np.abs(v)
            peak[s, h] = (p * vs).max()
            top[s, h] = np.abs(x).max()
    return out, spread, peak, top
