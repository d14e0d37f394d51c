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
