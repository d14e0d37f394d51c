"""CPU oracle of the paged 8-bit key/value cache, in 64 bits (numpy): block
tables and slot maps, the quantising append, the read-back and the attention
over the cache.  Shares no code with the CUDA path; written block by block and
row by row from the definitions."""
from __future__ import annotations

import math

import numpy as np

E4M3, INT8 = 0, 1
MOST = {E4M3: 448.0, INT8: 127.0}


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; exponent 0 is subnormal; all ones is NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if c & 127 == 127 else -v if c & 128 else v
    return out


_E4 = e4m3_values()


def decode_codes(code: int, raw: np.ndarray) -> np.ndarray:
    """Values of raw bytes (uint8)."""
    return _E4[raw] if code == E4M3 else raw.astype(np.uint8).view(np.int8).astype(np.float64)


def encode(code: int, y: np.ndarray) -> np.ndarray:
    """Nearest code of each finite value, ties to even, saturating: uint8."""
    y = np.asarray(y, np.float64)
    if code == INT8:
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(y), 448.0)
    exp = np.floor(np.log2(np.maximum(a, 2.0 ** -6))).astype(int)
    step = np.ldexp(1.0, exp - 3)
    v = np.rint(a / step) * step                       # np.rint: half to even
    v = np.minimum(v, 448.0)
    pos = _E4[:127]                                    # 0 .. 448, ascending
    c = np.searchsorted(pos, v).astype(np.uint8)
    assert np.array_equal(pos[c], v)
    return np.where(np.signbit(y), c | 128, c).astype(np.uint8)


def scale_for(code: int, amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= M s."""
    e = -126
    while amax > MOST[code] * math.ldexp(1.0, e):
        e += 1
    return math.ldexp(1.0, e)


def tables(cur, want, free, n_free, table, block, tokens):
    """(n_free, table, free, cu, slot) after the step, or None when refused."""
    cur, want, free, table = list(cur), list(want), list(free), np.array(table)
    pages, cap = len(free), table.shape[1] * block
    if any(not 0 <= x <= cap for x in cur + want) or not 0 <= n_free <= pages:
        return None
    nb = lambda x: -(-x // block)  # noqa: E731
    stack = free[:n_free]
    for b, (c, w) in enumerate(zip(cur, want)):
        stack += [int(table[b, j]) for j in range(nb(w), nb(c))]
    if sum(max(0, nb(w) - nb(c)) for c, w in zip(cur, want)) > len(stack):
        return None
    if sum(max(0, w - c) for c, w in zip(cur, want)) > tokens:
        return None
    cu, slot = [0], []
    for b, (c, w) in enumerate(zip(cur, want)):
        for j in range(nb(c), nb(w)):
            table[b, j] = stack.pop()
        slot += [int(table[b, t // block]) * block + t % block for t in range(c, w)]
        cu.append(len(slot))
    return len(stack), table, stack + free[len(stack):], cu, slot + [-1] * (tokens - len(slot))


def append(code, block, K, slot, codes, scale):
    """Appends one tensor: K [tokens, Hkv, d] into raw codes [pages, Hkv,
    block, d] (uint8) and scales [pages, Hkv], in place; returns the touched
    (page, rows held) of each run."""
    i, runs = 0, []
    while i < len(slot):
        if slot[i] < 0:
            i += 1
            continue
        j = i + 1
        while j < len(slot) and slot[j] == slot[j - 1] + 1 and slot[j] % block:
            j += 1
        page, off = slot[i] // block, slot[i] % block
        runs.append((i, j, page, off))
        for h in range(K.shape[1]):
            x = K[i:j, h].astype(np.float64)
            fin = np.where(np.isfinite(x), np.abs(x), 0.0)
            amax, was = float(fin.max()), float(scale[page, h])
            now = was if off > 0 and was > 0 and amax <= MOST[code] * was else scale_for(code, amax)
            if off > 0 and now != was:
                codes[page, h, :off] = encode(code, decode_codes(code, codes[page, h, :off]) * (was / now))
            y = np.where(np.isnan(x), 0.0, np.clip(x / now, -MOST[code], MOST[code]))
            codes[page, h, off:off + j - i] = encode(code, y)
            scale[page, h] = now
        i = j
    return runs


def values(code, codes, scale):
    """[pages, Hkv, block, d] values of a cache."""
    return decode_codes(code, codes) * scale.astype(np.float64)[..., None, None]


def rows_of(vals, table_row, n, head, block):
    """The first n cached rows of one sequence and head: [n, d]."""
    out = [vals[table_row[j], head] for j in range(-(-n // block))]
    return np.concatenate(out)[:n] if out else np.zeros((0, vals.shape[-1]))


def attend(q, k, v, bias):
    """One row: (o, lse, sum p |v|, largest sum |q k|); empty: zeros, -inf."""
    if not len(k) or np.all(np.isneginf(bias)):
        return np.zeros(v.shape[-1] if v.ndim == 2 else len(q)), -np.inf, np.zeros(len(q)), 0.0
    z = k @ q + bias
    m = z.max()
    p = np.exp(z - m)
    l = p.sum()
    return p @ v / l, m + math.log(l), p @ np.abs(v) / l, float((np.abs(k) @ np.abs(q)).max())


def decode_row(q, kvals, vvals, table_row, n, head, block, flags, idx=None, score=None):
    """One query head of a decode (flags: 1 sink, 2 local, 4 gate, 8 hier)."""
    k, v = (rows_of(x, table_row, n, head, block) for x in (kvals, vvals))
    local = -(-n // block) - 1
    if idx is None:
        return attend(q, k, v, np.zeros(n))
    keep = [int(j) for j in idx if j >= 0] if n > 0 else []
    if not keep:
        return attend(q, k[:0], v[:0], np.zeros(0))
    sc = [float(x) for x in score[:len(keep)]]
    if flags & 8:
        parts = [attend(q, k[j * block:(j + 1) * block], v[j * block:(j + 1) * block],
                        np.zeros(len(k[j * block:(j + 1) * block]))) for j in keep]
        w = np.exp(np.array(sc) - max(sc))
        lse = max(sc) + math.log(w.sum())
        w /= w.sum()
        return (sum(x * y[0] for x, y in zip(w, parts)), lse, sum(x * y[2] for x, y in zip(w, parts)),
                max(y[3] for y in parts))
    at = np.concatenate([np.arange(j * block, min(n, (j + 1) * block)) for j in keep])
    bias = []
    for j, s in zip(keep, sc):
        forced = (j == local and flags & 2) or (j == 0 and flags & 1)
        x = s - sc[-1]
        gate = 0.0 if forced or not flags & 4 else min(x, 0.0) - math.log1p(math.exp(-abs(x)))
        bias += [gate] * (min(n, (j + 1) * block) - j * block)
    return attend(q, k[at], v[at], np.array(bias))
