"""The paged 8-bit cache where it can go wrong without a large error: weights
far below the largest one, value scales far apart, ranges of many steps, rows
that one key decides, scales that are no powers of two.

Tolerances, per output element, with A = sum p |v| / sum p and Z the largest
scale * sum |q k| over the row's keys: the output is rounded once; the bf16
kernels round a weight to fp16 (half a step, 2^-11 of it), and one that falls
below fp16's normal range is off by 2^-32 of the row's largest weight at most
(`floor`); logits are fp32 sums of d products, d 2^-24 Z off at most, and pass
an exponential good to 2^-22; sums of n weights in fp32 add n 2^-24.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import block_sparse_long_landmark_b200 as sa
from oracle import paged as op
from test_gpu_paged import T, done, i32, random_table, raw

pytestmark = pytest.mark.gpu


def check_close(dtype, got, got_lse, ref, n, d, floor, what):
    """A row against the oracle's (o, lse, A, Z)."""
    o, lse, A, Z = ref
    got = got.double().cpu().numpy()
    e = 2 * (d * 2.0 ** -24 * Z + 2.0 ** -22) + n * 2.0 ** -24
    tol = torch.finfo(T[dtype]).eps / 2 * np.abs(o) + ((2.0 ** -11 if dtype == "bf16" else 0.0) + e) * A + floor
    bad = np.abs(got - o) > tol
    assert not bad.any(), (what, got[bad][:4], o[bad][:4], (np.abs(got - o) / tol).max())
    assert abs(float(got_lse) - lse) <= d * 2.0 ** -24 * Z + 2.0 ** -22 * (2 + abs(lse)) + n * 2.0 ** -24, (what, float(got_lse), lse)


def cache_of(p, codes, scales):
    ct = torch.float8_e4m3fn if p.code == op.E4M3 else torch.int8
    return tuple(torch.from_numpy(x).cuda().view(ct) for x in codes) + tuple(
        torch.from_numpy(x.astype(np.float32)).cuda() for x in scales)


# tokens of one sequence of a group of four heads: 8 rows a kv-head go through
# the decode's steps, 240 through the tiles
ROWS, TILES = 2, 60


# ---- weights far below the largest ---------------------------------------------------

def sink_row(p, code, n, bits, seed):
    """Codes, scales and queries [heads, d] with one key whose weight is 2^bits
    times the others' and whose value is zero."""
    rng = np.random.default_rng(seed)
    shape = (p.pages, p.Hkv, p.block, p.d)
    K = np.zeros(shape)
    K[..., 0][0, 0, 5] = 64.0
    K[..., 1:] = rng.integers(-15, 16, shape[:3] + (p.d - 1,))
    V = rng.integers(-100, 101, shape).astype(float)
    V[0, 0, 5] = 0.0
    codes = [op.encode(p.code, x) for x in (K, V)]
    ks, vs = np.full(shape[:2], 1.0 / 64), np.full(shape[:2], 0.01)
    q = np.zeros((p.Hq, p.d))
    q[:, 1:] = rng.standard_normal((p.Hq, p.d - 1)) * 0.4
    q[:, 0] = bits * math.log(2.0) * p.d ** 0.5
    return codes, (ks, vs), q


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("bits", [16, 20, 24, 27])
@pytest.mark.parametrize("form,n", [("decode", 128), ("decode", 1000), ("kept", 128), ("hier", 256), ("rows", 128),
                                    ("rows", 1000), ("tiles", 128), ("tiles", 1000)])
def test_weights_far_below_the_largest(form, n, bits, code):
    """A key that takes nearly all the weight and has no value (a sink): what is
    left of the row comes from weights 2^-16 to 2^-27 of the largest."""
    d, block, Hq = 64, 64, 4
    maxb = -(-n // block)
    tokens = {"rows": ROWS, "tiles": TILES}.get(form, 0)
    flags = {"kept": sa.SA_SINK | sa.SA_LOCAL, "hier": sa.SA_SINK | sa.SA_LOCAL | sa.SA_HIER}.get(form, 0)
    p = sa.make_paged_params(1, Hq, 1, d, block, maxb, maxb, tokens, 8, flags, code=code)
    codes, scales, q = sink_row(p, code, n, bits, n + bits)
    idx = sc = lists = None
    if form in ("kept", "hier"):
        idx, sc = np.full(10, -1, np.int32), np.zeros(10, np.float32)
        idx[:maxb] = range(maxb)
        if form == "hier":
            q[:, 0] = 0                        # the block decides, not the key
            codes[1][0] = 0                    # and its values are zero
            sc[0] = bits * math.log(2.0)
        lists = (i32(idx.tolist()), torch.from_numpy(sc).cuda(), i32([maxb]))
    cache = cache_of(p, codes, scales)
    vals = [op.values(p.code, c, s.astype(np.float32)) for c, s in zip(codes, scales)]
    table, ws = np.arange(maxb, dtype=np.int32)[None], sa.paged_workspace(p)
    Q = torch.from_numpy(q).bfloat16()
    if tokens:
        Q = Q.repeat(tokens, 1, 1)
        Q[..., 1:] *= 1 + torch.arange(tokens)[:, None, None] / 64
        O, lse = sa.paged_prefill(p, Q.cuda(), i32([0, tokens]), cache, i32(table.tolist()), i32([n]), ws)
        O, lse = O[::7], lse[::7]
        Q = Q[::7]
    else:
        O, lse = sa.paged_decode(p, Q[None].contiguous().cuda(), cache, i32(table.tolist()), i32([n]), ws, lists=lists)
        Q = Q[None]
    done(ws)
    floor = 2.0 ** -32 * np.abs(vals[1]).sum((0, 1, 2))
    for t in range(len(Q)):
        for h in (0, 3):
            ref = op.decode_row(Q[t, h].double().numpy() * d ** -0.5, *vals, table[0], n, 0, block, flags, idx, sc)
            check_close("bf16", O[t, h], lse[t, h], ref, n, d, floor, (t, h))


# ---- value scales far apart -------------------------------------------------------------

@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("n,where", [(300, "first"), (300, "last"), (300, "all"), (1500, "first"), (1500, "middle")])
@pytest.mark.parametrize("tokens", [ROWS, TILES])
def test_value_scales_of_zero_and_far_apart(tokens, n, where, code):
    """Pages with a value scale of 0 at either end and all over, the others
    spread over 2^60; tiny and huge queries."""
    d, block, Hq = 128, 32, 4
    maxb = -(-n // block)
    p = sa.make_paged_params(1, Hq, 1, d, block, maxb, maxb, tokens, flags=sa.SA_CAUSAL, code=code)
    rng = np.random.default_rng(n)
    codes = [op.encode(p.code, rng.standard_normal((maxb, 1, block, d)) * 40) for _ in "kv"]
    ks, vs = rng.uniform(1e-4, 3e-3, (maxb, 1)), 2.0 ** rng.uniform(-30, 30, (maxb, 1))
    vs[{"first": slice(0, 5), "last": slice(maxb - 5, maxb), "all": slice(0, maxb), "middle": slice(9, 20)}[where]] = 0
    ks, vs = ks.astype(np.float32), vs.astype(np.float32)
    cache = cache_of(p, codes, (ks, vs))
    Q = torch.from_numpy(rng.standard_normal((tokens, Hq, d)) * 2.0 ** rng.integers(-4, 5, (tokens, Hq, 1)))
    Q[0, 0] *= 2.0 ** -100
    Q[0, 1] *= 2.0 ** 8
    Q = Q.bfloat16()
    ws = sa.paged_workspace(p)
    O, lse = sa.paged_prefill(p, Q.cuda(), i32([0, tokens]), cache, i32([list(range(maxb))]), i32([n]), ws)
    done(ws)
    kv = [op.values(p.code, c, s) for c, s in zip(codes, (ks, vs))]
    for t in {0, 1, tokens // 2, tokens - 1}:
        see = n - tokens + t + 1
        for h in range(Hq):
            q = Q[t, h].double().numpy() * d ** -0.5
            ref = op.decode_row(q, *kv, list(range(maxb)), see, 0, block, 0)
            # the tiles round a weight times its value's scale
            floor = 2.0 ** -32 * float(vs.max()) * np.abs(op.decode_codes(p.code, codes[1])).sum((0, 1, 2))
            check_close("bf16", O[t, h], lse[t, h], ref, see, d, floor, (t, h))


@pytest.mark.parametrize("bits,up,zero", [(60, 40, -60), (110, 40, -100), (120, 60, -126), (20, 60, 0), (115, 90, -40)])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_tiles_join_what_value_scales_set_apart(code, bits, up, zero):
    """A block of no value takes the weight (its scale is tiny, or 0), and what
    lies 2^bits below has values of scale 2^up: the row is what that leaves."""
    n, d, block, Hq, tokens = 192, 64, 64, 4, TILES
    p = sa.make_paged_params(1, Hq, 1, d, block, 3, 3, tokens, code=code)
    codes, (ks, vs), q = sink_row(p, code, n, bits, 3)
    vs[:] = 2.0 ** up
    codes[1][0] = 0
    vs[0] = 2.0 ** zero if zero else 0.0
    cache = cache_of(p, codes, (ks, vs))
    Q = torch.from_numpy(q).bfloat16().repeat(tokens, 1, 1)
    ws = sa.paged_workspace(p)
    O, lse = sa.paged_prefill(p, Q.cuda(), i32([0, tokens]), cache, i32([[0, 1, 2]]), i32([n]), ws)
    done(ws)
    kv = [op.values(p.code, c, s.astype(np.float32)) for c, s in zip(codes, (ks, vs))]
    raws = op.decode_codes(p.code, codes[1])[:, 0].reshape(-1, d)
    for t, h in ((0, 0), (33, 1), (tokens - 1, 3)):
        qd = Q[t, h].double().numpy() * d ** -0.5
        ref = op.decode_row(qd, *kv, [0, 1, 2], n, 0, block, 0)
        z = kv[0][:, 0].reshape(-1, d) @ qd
        w = np.exp(z - z.max()) * np.repeat(vs[:, 0], block)
        floor = 2.0 ** -32 * w.max() * np.abs(raws).sum(0)        # a weight times its value's scale is what is rounded
        check_close("bf16", O[t, h], lse[t, h], ref, n, d, floor, (t, h))
