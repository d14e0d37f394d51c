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


# ---- ranges of many steps ------------------------------------------------------------------

def pooled_cache(p, seed):
    """A cache of drawn codes, quickly made, with scales that differ."""
    rng = np.random.default_rng(seed)
    pool = op.encode(p.code, rng.standard_normal(1 << 16) * (60 if p.code == op.E4M3 else 30))
    shape = (p.pages, p.Hkv, p.block, p.d)
    codes = [pool[rng.integers(0, 1 << 16, shape)] for _ in "kv"]
    scales = [rng.uniform(0.004, 0.03, shape[:2]).astype(np.float32) for _ in "kv"]
    return cache_of(p, codes, scales), [op.values(p.code, c, s) for c, s in zip(codes, scales)]


def sms():
    return min(148, torch.cuda.get_device_properties(0).multi_processor_count)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("code,d,block,Hq,Hkv", [("e4m3", 128, 64, 32, 8), ("int8", 128, 48, 40, 8),
                                                 ("int8", 64, 16, 24, 8), ("e4m3", 64, 128, 32, 8)])
def test_tiles_of_many_steps(code, d, block, Hq, Hkv, causal):
    """Every CTA walks through twenty key tiles and more, units of one and of
    two query tiles after one another; the pages are shared, as they may be."""
    lens, grown = [9000, 16000, 12345, 100, 9999], [300, 2048, 30, 72, 33]
    G, maxb = Hq // Hkv, -(-16000 // block)
    tpu = 2 * (128 // G)
    tiles = sum(-(-(min(n, n - g + min(g, t + tpu)) if causal else n) // 128) for n, g in zip(lens, grown) for t in range(0, g, tpu))
    assert tiles * Hkv >= 20 * sms() and any(0 < g % tpu <= tpu // 2 for g in grown)
    cu = [sum(grown[:i]) for i in range(6)]
    p = sa.make_paged_params(5, Hq, Hkv, d, block, 150, maxb, cu[-1] + 3, flags=sa.SA_CAUSAL if causal else 0, code=code)
    cache, kv = pooled_cache(p, 1)
    rng = np.random.default_rng(2)
    table = rng.integers(0, p.pages, (5, maxb)).astype(np.int32)
    Q = torch.from_numpy(rng.standard_normal((p.tokens, Hq, d)) * rng.choice([1.0, 6.0], (p.tokens, Hq, 1))).bfloat16()
    ws = sa.paged_workspace(p)
    O, lse = sa.paged_prefill(p, Q.cuda(), i32(cu), cache, i32(table.tolist()), i32(lens), ws)
    done(ws)
    for b, (n, g) in enumerate(zip(lens, grown)):
        for t in sorted({0, 63, g // 3, g // 2, g - 65, g - 1} & set(range(g))):
            for h in (t % Hq, (t + 5 * b + 9) % Hq):
                see = n - g + t + 1 if causal else n
                ref = op.decode_row(Q[cu[b] + t, h].double().numpy() * d ** -0.5, *kv, table[b], see, h // G, block, 0)
                floor = 2.0 ** -32 * np.abs(op.rows_of(kv[1], table[b], see, h // G, block)).sum(0)
                check_close("bf16", O[cu[b] + t, h], lse[cu[b] + t, h], ref, see, d, floor, (b, t, h))


@pytest.mark.parametrize("form", ["decode", "rows"])
@pytest.mark.parametrize("code,d,block,Hq,Hkv", [("e4m3", 128, 64, 32, 8), ("int8", 128, 16, 32, 8),
                                                 ("int8", 64, 112, 80, 8), ("e4m3", 64, 32, 16, 8)])
def test_steps_of_many_stages(code, d, block, Hq, Hkv, form):
    """Every warp streams thirty stages and more: more than one batch of parts,
    every place of the stage memory used again and again."""
    B = 32
    lens = [16000 - 97 * b for b in range(B)]
    G, maxb = Hq // Hkv, -(-16000 // block)
    grown = [1 + b % 3 for b in range(B)]
    T_ = sum(grown) if form == "rows" else 0
    assert sum(-(-n // 64) for n in lens) * Hkv >= 30 * sms() * 12
    p = sa.make_paged_params(B, Hq, Hkv, d, block, 150, maxb, T_, flags=sa.SA_CAUSAL, code=code)
    cache, kv = pooled_cache(p, 1)
    rng = np.random.default_rng(2)
    table = rng.integers(0, p.pages, (B, maxb)).astype(np.int32)
    cu = [sum(grown[:i]) for i in range(B + 1)]
    Q = torch.from_numpy(rng.standard_normal((T_ or B, Hq, d)) * 2.0 ** rng.integers(-1, 3, (T_ or B, Hq, 1))).bfloat16()
    ws = sa.paged_workspace(p)
    args = cache, i32(table.tolist()), i32(lens), ws
    O, lse = sa.paged_prefill(p, Q.cuda(), i32(cu), *args) if T_ else sa.paged_decode(p, Q.cuda(), *args)
    done(ws)
    for b in range(0, B, 3):
        for t in range(grown[b] if T_ else 1):
            for h in ((b + t) % Hq, (b + 7 * t + 11) % Hq):
                row, see = (cu[b] + t, lens[b] - grown[b] + t + 1) if T_ else (b, lens[b])
                ref = op.decode_row(Q[row, h].double().numpy() * d ** -0.5, *kv, table[b], see, h // G, block, 0)
                floor = 2.0 ** -32 * np.abs(op.rows_of(kv[1], table[b], see, h // G, block)).sum(0)
                check_close("bf16", O[row, h], lse[row, h], ref, see, d, floor, (b, t, h))


# ---- one value row decides ---------------------------------------------------------------------

@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("tokens,d,block", [(0, 128, 64), (0, 64, 112), (0, 128, 16), (ROWS, 64, 48), (ROWS, 128, 128),
                                            (TILES, 128, 64), (TILES, 64, 48), (TILES, 128, 16), (TILES, 64, 128)])
def test_one_value_row_decides(tokens, d, block, code):
    """All values but one key's are zero, for keys at the ends of tiles, pages
    and the sequence: a row in the wrong place, or a wrong scale, is the whole output."""
    n, Hq = 5 * 128 + 37, 4
    keys = sorted({0, 15, 16, 63, 64, 127, 128, 255, 256, 383, 575, 576, 639, 640, n - 6, n - 1, block - 1, block,
                   n // block * block - 1, n // block * block})
    maxb, B = -(-n // block), len(keys)
    p = sa.make_paged_params(B, Hq, 1, d, block, B * maxb, maxb, tokens * B, code=code)
    cache, kv = pooled_cache(p, 4)
    table = random_table(p, [n] * B, 4)
    vals = raw(cache[1])
    keep = np.zeros(vals.shape, bool)
    for b, j in enumerate(keys):
        keep[table[b, j // block], 0, j % block] = True
    vals[~keep] = 0
    cache = (cache[0], torch.from_numpy(vals).cuda().view(cache[1].dtype), *cache[2:])
    kv[1] = op.values(p.code, vals, cache[3].cpu().numpy())
    Q = torch.from_numpy(np.random.default_rng(3).standard_normal((tokens * B or B, Hq, d)) / 3).bfloat16()
    ws = sa.paged_workspace(p)
    args = cache, i32(table.tolist()), i32([n] * B), ws
    if tokens:
        O, lse = sa.paged_prefill(p, Q.cuda(), i32([tokens * b for b in range(B + 1)]), *args)
    else:
        O, lse = sa.paged_decode(p, Q.cuda(), *args)
    done(ws)
    for b in range(B):
        for t in {0, tokens // 2, tokens - 1} if tokens else {0}:
            row = b * max(1, tokens) + t
            ref = op.decode_row(Q[row, 1].double().numpy() * d ** -0.5, *kv, table[b], n, 0, block, 0)
            check_close("bf16", O[row, 1], lse[row, 1], ref, n, d, 2.0 ** -32 * np.abs(kv[1]).max((0, 1, 2)), (keys[b], t))


# ---- queries that are not numbers, block by block -------------------------------------------

@pytest.mark.parametrize("dtype,block", [("bf16", 64), ("bf16", 16), ("bf16", 128), ("fp32", 64)])
def test_hierarchical_decode_keeps_a_query_that_is_not_a_number(dtype, block):
    """Its row's output is NaN, its lse the lists' alone; other rows are untouched."""
    lens, maxb = [500, 321], -(-500 // block)
    p = sa.make_paged_params(2, 8, 2, 128, block, 2 * maxb, maxb, 0, 3, sa.SA_SINK | sa.SA_LOCAL | sa.SA_HIER, dtype)
    cache, _ = pooled_cache(p, 2)
    table, n, ws = i32(random_table(p, lens, 2).tolist()), i32(lens), sa.paged_workspace(p)
    idx, cnt = i32([[[0, 1, -(-m // block) - 1, -1, -1]] * 2 for m in lens]), i32([[3, 3]] * 2)
    sc = torch.randn(2, 2, 5, device="cuda")
    q = torch.randn(2, 8, 128, device="cuda").to(T[dtype])
    bad = q.clone()
    bad[0, 3, 7], bad[1, 0, 0] = math.nan, math.inf
    o, lse = sa.paged_decode(p, q, cache, table, n, ws, lists=(idx, sc, cnt))
    o2, lse2 = sa.paged_decode(p, bad, cache, table, n, ws, lists=(idx, sc, cnt))
    done(ws)
    keep = torch.ones(2, 8, dtype=torch.bool, device="cuda")
    keep[0, 3] = keep[1, 0] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert torch.isnan(o2[~keep].float()).all() and not torch.isnan(o.float()).any()
    assert torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,block", [("bf16", 64), ("bf16", 128), ("fp32", 16)])
@pytest.mark.parametrize("where", [[0], [1], [2], [0, 1], [0, 1, 2]])
def test_hierarchical_blocks_of_no_weight(dtype, block, where):
    """A block whose score is -inf takes no part, the first ones and all of them too."""
    n, maxb = 500, -(-500 // block)
    p = sa.make_paged_params(1, 4, 1, 128, block, maxb, maxb, 0, 3, sa.SA_SINK | sa.SA_LOCAL | sa.SA_HIER, dtype)
    cache, kv = pooled_cache(p, 2)
    table, ws = random_table(p, [n], 2), sa.paged_workspace(p)
    idx, sc = [0, 1, maxb - 1, -1, -1], np.zeros(5, np.float32)
    sc[:3] = [0.3, -1.0, 2.0]
    sc[where] = -math.inf
    q = torch.randn(1, 4, 128, device="cuda").to(T[dtype])
    o, lse = sa.paged_decode(p, q, cache, i32(table.tolist()), i32([n]), ws,
                             lists=(i32([[idx]]), torch.from_numpy(sc).cuda()[None, None], i32([[3]])))
    done(ws)
    live = [i for i in range(3) if i not in where]
    if not live:
        assert not o.any() and torch.isneginf(lse).all()
        return
    for h in range(4):
        ref = op.decode_row(q[0, h].double().cpu().numpy() * 128 ** -0.5, *kv, table[0], n, 0, block, p.flags,
                            [idx[i] for i in live], sc[live])
        check_close(dtype, o[0, h], lse[0, h], ref, n, 128, 2.0 ** -32 * np.abs(kv[1]).sum((0, 1, 2)), h)


# ---- a flag that only lists have a use for -------------------------------------------------

@pytest.mark.parametrize("dtype,d,block,Hq,Hkv", [("bf16", 128, 64, 32, 8), ("bf16", 64, 16, 40, 2), ("bf16", 128, 128, 24, 1),
                                                  ("fp32", 64, 32, 8, 2)])
def test_dense_decode_of_lists_per_query_head(dtype, d, block, Hq, Hkv):
    """Without lists, SA_SELECT_PER_QHEAD changes nothing: a kv-head's query
    heads read its cache together, in the same order of sums."""
    lens = [9000, 5, 0, 2500]
    maxb = -(-9000 // block)
    a, b = (sa.make_paged_params(4, Hq, Hkv, d, block, 200, maxb, flags=f, dtype=dtype) for f in (0, sa.SA_SELECT_PER_QHEAD))
    cache, _ = pooled_cache(a, 2)
    table = i32(np.random.default_rng(1).integers(0, 200, (4, maxb)).tolist())
    q = torch.randn(4, Hq, d, device="cuda").to(T[dtype])
    out = []
    for p in (a, b):
        ws = sa.paged_workspace(p, ops=[sa.SA_OP_PAGED_DECODE])
        out.append(sa.paged_decode(p, q, cache, table, i32(lens), ws))
        done(ws)
    assert all(torch.equal(x, y) for x, y in zip(*out))


# ---- which kernel a chunk call runs ----------------------------------------------------------

def launches_of(B, tokens, Hq, Hkv, block, max_blocks, grown, lens):
    p = sa.make_paged_params(B, Hq, Hkv, 128, block, 64, max_blocks, tokens, flags=sa.SA_CAUSAL)
    cache, kv = pooled_cache(p, 2)
    table = np.random.default_rng(1).integers(0, 64, (B, max_blocks)).astype(np.int32)
    cu = [sum(grown[:i]) for i in range(B + 1)]
    Q = torch.randn(tokens, Hq, 128, dtype=torch.float32).bfloat16()
    ws = sa.paged_workspace(p, ops=[sa.SA_OP_PAGED_PREFILL])
    torch.cuda.synchronize()
    n = sa.sparse_attn_launch_count()
    O, lse = sa.paged_prefill(p, Q.cuda(), i32(cu), cache, i32(table.tolist()), i32(lens), ws)
    n = sa.sparse_attn_launch_count() - n
    done(ws)
    for b in range(B):
        for t in {0, grown[b] - 1} & set(range(grown[b])):
            see, h = lens[b] - grown[b] + t + 1, (b + t) % Hq
            ref = op.decode_row(Q[cu[b] + t, h].double().numpy() * 128 ** -0.5, *kv, table[b], see, h // (Hq // Hkv), block, 0)
            floor = 2.0 ** -32 * np.abs(op.rows_of(kv[1], table[b], see, h // (Hq // Hkv), block)).sum(0)
            check_close("bf16", O[cu[b] + t, h], lse[cu[b] + t, h], ref, see, 128, floor, (b, t, h))
    return n


@pytest.mark.parametrize("B,grown", [(2, [63, 1]), (2, [0, 63]), (65, [192] + [1] * 64), (128, [897] + [1] * 127)])
def test_a_long_chunk_beside_single_tokens_goes_to_the_tiles(B, grown):
    """Tables for 128K keys: a chunk's rows, hidden in a call of few rows, are
    not taken 8 or 16 at a time over its whole cache."""
    G = 1 if B == 128 else 4
    lens = [max(1000, grown[0] + 100)] + [300 + b for b in range(1, B)]
    assert launches_of(B, sum(grown), 2 * G, 2, 64, 2048, grown, lens) == 5


@pytest.mark.parametrize("B,grown,max_blocks", [(2, [5, 5], 2048), (8, [5] * 8, 79), (64, [1] * 64, 4)])
def test_few_rows_stay_in_the_decodes_steps(B, grown, max_blocks):
    """Up to 40 rows in all, or what a hidden chunk can read again is little."""
    assert launches_of(B, sum(grown), 8, 2, 64, max_blocks, grown, [200 + b % 50 for b in range(B)]) == 2


# ---- scales of other makers ----------------------------------------------------------------

@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_append_to_subnormal_scales(code, few):
    """What a page holds at a scale under 2^-126 is kept, or rounded anew to the scale that grows."""
    pages, Hkv, d, block, held = (6, 2, 64, 32, 7) if few else (6 * 200, 8, 64, 32, 7)
    p = sa.make_paged_params(pages, Hkv, Hkv, d, block, pages, 1, 2 * pages, code=code, dtype="fp32")
    assert (2 * p.tokens * Hkv <= 64 * sms()) == few
    rng = np.random.default_rng(5)
    codes = [op.encode(p.code, rng.standard_normal((pages, Hkv, block, d)) * 40) for _ in "kv"]
    scale = [np.resize([2.0 ** -127, 2.0 ** -130, 2.0 ** -133 * 5], (pages, Hkv)) for _ in "kv"]
    x = [rng.choice([0.0, 2.0 ** -125, 2.0 ** -122, 2.0 ** -120], (pages, 1, 1, 1)) * rng.choice([0, 1, -1], (pages, 2, Hkv, d)) for _ in "kv"]
    x = [y.reshape(2 * pages, Hkv, d) for y in x]
    cache, ws = cache_of(p, codes, scale), sa.paged_workspace(p)
    assert all(np.array_equal(c.double().cpu().numpy(), s) for c, s in zip(cache[2:], scale))
    slot = [b * block + held + i for b in range(pages) for i in range(2)]
    sa.paged_append(p, *(torch.from_numpy(y.astype(np.float32)).cuda() for y in x), torch.tensor(slot, device="cuda"), cache, ws)
    done(ws)
    for i in range(2):
        was = scale[i].copy()
        op.append(p.code, block, x[i], slot, codes[i], scale[i])
        assert 0 < (scale[i] != was).mean() < 1
        assert np.array_equal(cache[2 + i].double().cpu().numpy(), scale[i]), i
        assert np.array_equal(raw(cache[i]), codes[i]), i

def near_tie_scales(code, rng, n):
    """fp32 scales below 1 and, for each, a code c such that c * scale is next
    to a border between two codes of scale 1."""
    t, c = (rng.choice(np.arange(8, 16) + 0.5, n), 2 * rng.integers(8, 16, n)) if code == "e4m3" else (
        rng.choice(np.arange(0, 60) + 0.5, n), rng.integers(65, 128, n))
    return (t / c).astype(np.float32), c


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 64), ("fp32", 64, 32), ("fp32", 128, 128), ("bf16", 64, 16)])
def test_append_to_scales_that_are_no_powers_of_two(dtype, d, block, code, few):
    """Pages filled elsewhere: a scale that is kept divides the new rows, one
    that grows is divided by a power of two, and either is one rounding, next
    to the border between two codes too; one old scale is 0."""
    rng = np.random.default_rng(d + block)
    pages, Hkv = (8, 2) if few else (600, 8)
    held, new = 5, 3
    p = sa.make_paged_params(pages, Hkv, Hkv, d, block, pages, 1, pages * new, dtype=dtype, code=code)
    assert (2 * p.tokens * Hkv <= 64 * sms()) == few
    M, c8 = op.MOST[p.code], p.code
    codes, scale, x = [], [], []
    for _ in "kv":
        raw8 = op.encode(c8, rng.standard_normal((pages, Hkv, block, d)) * 30)
        s, c = near_tie_scales(code, rng, pages * Hkv)
        s, c = s.reshape(pages, Hkv), c.reshape(pages, Hkv)
        raw8[..., :held, :8] = op.encode(c8, c[..., None, None].astype(float))
        # heads in turn: kept, grown, kept, grown
        y = rng.standard_normal((pages, new, Hkv, d))
        for h in range(Hkv):
            if h % 2 == 0:
                ties = rng.choice(np.arange(8, 16) + 0.5 if code == "e4m3" else np.arange(0, 100) + 0.5, (pages, new, d))
                y[:, :, h] = ties * s[:, h, None, None].astype(np.float64) * rng.choice([1, -1], (pages, new, d))
            else:
                y[:, :, h] = np.clip(y[:, :, h], -3.5, 3.5)
                y[:, 0, h, 0] = M                                # the scale becomes 1
        s[1, 0] = 0.0
        codes.append(raw8)
        scale.append(s.astype(np.float64))
        x.append(torch.from_numpy(y.reshape(pages * new, Hkv, d)).to(T[dtype]))
    cache, ws = cache_of(p, codes, scale), sa.paged_workspace(p)
    slot = [page * block + held + i for page in range(pages) for i in range(new)]
    L = torch.zeros(pages, Hkv, 1, d, dtype=T[dtype], device="cuda")
    sa.paged_append(p, x[0].cuda(), x[1].cuda(), torch.tensor(slot, device="cuda"), cache, ws,
                    cu=i32([new * b for b in range(pages + 1)]), new_len=i32([held + new] * pages), L=L)
    done(ws)
    grown = 0
    for i in range(2):
        was = scale[i].copy()
        op.append(c8, block, x[i].double().numpy(), slot, codes[i], scale[i])
        grown += (scale[i] != was).sum()
        assert np.array_equal(cache[2 + i].double().cpu().numpy(), scale[i]), i
        got = raw(cache[i])
        assert np.array_equal(got, codes[i]), (i, (got != codes[i]).sum())
    assert 0.4 < grown / (2 * pages * Hkv) < 0.6
    ref = op.values(c8, codes[0], scale[0])[:, :, :held + new].mean(2)
    tol = (torch.finfo(T[dtype]).eps / 2 + 3 * 2.0 ** -24) * np.abs(ref) + 2.0 ** -24 * M * scale[0][..., None]
    assert (np.abs(L[:, :, 0].double().cpu().numpy() - ref) <= tol).all()


# ---- pages given back -------------------------------------------------------------------------

@pytest.mark.parametrize("bad", [-1, 8, -2 ** 31, 2 ** 31 - 1])
def test_tables_report_a_bad_page_that_is_given_back(bad):
    """Where it is given back, not in the step that pops it."""
    p = sa.make_paged_params(2, 1, 1, 64, 16, 8, 4, 10)
    ws = sa.paged_workspace(p, ops=[sa.SA_OP_PAGED_TABLES])
    table = i32([[1, bad, 3, -1], [5, -1, -1, -1]])
    free, n_free = i32([0, 2, 4, 6, 7, 0, 0, 0]), i32([5])
    n, cu, slot = sa.paged_tables(p, i32([40, 3]), i32([10, 4]), free, n_free, table, ws)
    torch.cuda.synchronize()
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 1)
    assert n.item() == 7 and free[5:7].tolist() == [bad, 3] and slot.tolist() == [5 * 16 + 3] + [-1] * 9
    # behind a sequence's last block anything may stand
    n, cu, slot = sa.paged_tables(p, i32([10, 4]), i32([9, 5]), free, n, table, ws)
    done(ws)
