"""The paged 8-bit cache against its 64-bit oracle: block tables, append,
read-back, decode and chunked prefill, alone and as a captured step.

Tolerances of the attention, per output element, with A = sum p |v| / sum p and
Z the largest scale * sum |q k| over the row's keys (both from the oracle):
the output is rounded once (half a step of its type); the kernels may round
the softmax weights to bf16 (half a step, 2^-8, of each weight); the logits are
fp32 sums of d products, d 2^-24 Z off at most, and pass an exponential good to
2^-22; sums of n weights in fp32 add n 2^-24.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import block_sparse_long_landmark_b200 as sa
from oracle import paged as op

pytestmark = pytest.mark.gpu

CODE = {"e4m3": op.E4M3, "int8": op.INT8}
T = {"bf16": torch.bfloat16, "fp32": torch.float32}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def raw(t):
    return t.view(torch.uint8).cpu().numpy().copy()


def random_cache(p, seed, power_of_two=False):
    """Codes over the whole range (no NaN pattern) and scales that differ."""
    rng = np.random.default_rng(seed)
    shape = (p.pages, p.Hkv, p.block, p.d)
    c = []
    for _ in "kv":
        x = rng.standard_normal(shape) * (60 if p.code == op.E4M3 else 30)
        c.append(op.encode(p.code, x))
    sc = [(2.0 ** rng.integers(-8, -4, shape[:2]) if power_of_two else rng.uniform(0.004, 0.03, shape[:2])).astype(np.float32)
          for _ in "kv"]
    ct = torch.float8_e4m3fn if p.code == op.E4M3 else torch.int8
    cache = tuple(torch.from_numpy(x).cuda().view(ct) for x in c) + tuple(torch.from_numpy(x).cuda() for x in sc)
    return cache, c, sc


def random_table(p, lens, seed):
    rng = np.random.default_rng(seed)
    perm = list(rng.permutation(p.pages))
    t = np.full((p.B, p.max_blocks), -7, np.int32)     # behind a sequence: never read
    for b, n in enumerate(lens):
        for j in range(-(-n // p.block)):
            t[b, j] = perm.pop()
    return t


def tolerance(dtype, ref, A, Z, n, d):
    half = torch.finfo(T[dtype]).eps / 2
    e = 2 * (d * 2.0 ** -24 * Z + 2.0 ** -22) + n * 2.0 ** -24
    return half * np.abs(ref) + ((2.0 ** -8 if dtype == "bf16" else 0.0) + e) * A + 1e-30


def check_row(dtype, got, got_lse, ref, n, d, what):
    o, lse, A, Z = ref
    got = got.double().cpu().numpy()
    if np.isneginf(lse):
        assert np.isneginf(float(got_lse)) and not got.any(), what
        return
    bad = np.abs(got - o) > tolerance(dtype, o, A, Z, n, d)
    assert not bad.any(), (what, got[bad][:4], o[bad][:4])
    tol = d * 2.0 ** -24 * Z + 2.0 ** -22 * (2 + abs(lse)) + n * 2.0 ** -24
    assert abs(float(got_lse) - lse) <= tol, (what, float(got_lse), lse, tol)


def done(ws):
    torch.cuda.synchronize()
    assert sa.check_status(ws) == 0


# ---- block tables ---------------------------------------------------------------

def run_tables(p, cur, want, free, n_free, table):
    ws = sa.paged_workspace(p, ops=[sa.SA_OP_PAGED_TABLES])
    t, f = i32(table.tolist()), i32(free)
    out = sa.paged_tables(p, i32(cur), i32(want), f, i32([n_free]), t, ws)
    torch.cuda.synchronize()
    return ws, t.cpu().numpy(), f.cpu().tolist(), [x.cpu().numpy() for x in out]


@pytest.mark.parametrize("B,block,maxb,steps", [(1, 16, 3, 6), (7, 64, 9, 6), (300, 32, 5, 3), (2500, 16, 4, 2)])
def test_tables_follow_the_oracle(B, block, maxb, steps):
    rng = np.random.default_rng(B)
    pages = B * maxb + 3
    free, n_free = list(rng.permutation(pages)), pages
    table, cur = np.full((B, maxb), -1, np.int32), [0] * B
    for step in range(steps):
        want = [int(x) for x in rng.integers(0, maxb * block + 1, B)]
        if step % 2:
            want = [c if rng.random() < 0.5 else w for c, w in zip(cur, want)]
        tokens = sum(max(0, w - c) for c, w in zip(cur, want)) + (step * 5)
        p = sa.make_paged_params(B, 1, 1, 64, block, pages, maxb, tokens)
        ref = op.tables(cur, want, free, n_free, table, block, tokens)
        ws, t, f, (n, cu, slot) = run_tables(p, cur, want, free, n_free, table)
        assert sa.check_status(ws) == 0
        assert n[0] == ref[0] and list(cu) == ref[3] and list(slot) == ref[4]
        assert np.array_equal(t, ref[1]) and f[:ref[0]] == ref[2][:ref[0]]
        n_free, table, free, cur = int(n[0]), t, f, want


def test_tables_of_the_most_sequences():
    B, block, maxb = 16384, 16, 4
    rng = np.random.default_rng(0)
    want = [int(x) for x in rng.integers(0, maxb * block + 1, B)]
    pages = B * maxb
    free = list(rng.permutation(pages))
    table = np.full((B, maxb), -1, np.int32)
    p = sa.make_paged_params(B, 1, 1, 64, block, pages, maxb, sum(want))
    ref = op.tables([0] * B, want, free, pages, table, block, sum(want))
    ws, t, f, (n, cu, slot) = run_tables(p, [0] * B, want, free, pages, table)
    assert sa.check_status(ws) == 0
    assert n[0] == ref[0] and list(cu) == ref[3] and list(slot) == ref[4] and np.array_equal(t, ref[1])


@pytest.mark.parametrize("cur,want,n_free,tokens,bits", [
    ([0, 5], [40, 5], 2, 64, 16),           # three pages wanted, two free
    ([0, 5], [30, 5], 2, 29, 16),           # thirty slots wanted
    ([0, 5], [65, 5], 4, 100, 1),           # longer than the table
    ([0, -1], [4, 5], 4, 100, 1),
    ([0, 5], [4, -2], 4, 100, 1),
    ([0, 5], [4, 5], 9, 100, 1),            # more free pages than pages
    ([0, 5], [4, 5], -1, 100, 1),
])
def test_tables_refuse_as_a_whole(cur, want, n_free, tokens, bits):
    p = sa.make_paged_params(2, 1, 1, 64, 16, 8, 4, tokens)
    table = np.array([[1, 2, 3, 4], [5, 6, 7, 0]], np.int32)
    ws, t, f, (n, cu, slot) = run_tables(p, cur, want, list(range(8)), n_free, table)
    with pytest.raises(sa.SparseAttnError):
        sa.check_status(ws)
    ws, _, _, _ = run_tables(p, cur, want, list(range(8)), n_free, table)
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, bits)
    assert np.array_equal(t, table) and f == list(range(8)) and n[0] == n_free and not cu.any() and (slot == -1).all()


def test_tables_give_no_slot_on_a_bad_page():
    p = sa.make_paged_params(1, 1, 1, 64, 16, 4, 4, 40)
    ws, t, f, (n, cu, slot) = run_tables(p, [3], [20], [0, 9, 0, 0], 2, np.array([[77, -1, -1, -1]], np.int32))
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 1)
    assert (slot == -1).all() and t[0, 1] == -1 and cu[1] == 17


# ---- append and read-back ---------------------------------------------------------

def split_slots(p, table, lens, grown, pad=0):
    slot, cu = [], [0]
    for b, (n, k) in enumerate(zip(lens, grown)):
        slot += [int(table[b, t // p.block]) * p.block + t % p.block for t in range(n - k, n)]
        cu.append(len(slot))
    return slot + [-1] * pad, cu


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,d,block,Hkv", [("bf16", 128, 64, 2), ("bf16", 64, 16, 3), ("bf16", 128, 128, 1),
                                               ("fp32", 64, 48, 2), ("fp32", 128, 128, 2)])
def test_append_follows_the_oracle(code, dtype, d, block, Hkv):
    rng = np.random.default_rng(d + block)
    steps = [[1, 5, 0, 2 * block + 3, block], [1, block - 5, 3, 1, 1], [block, 1, 0, 200, block - 1]]
    B, maxb = 5, (500 // block) + 4
    lens = np.zeros(B, int)
    pages = B * maxb
    p0 = sa.make_paged_params(B, Hkv, Hkv, d, block, pages, maxb, 0, code=code, dtype=dtype)
    table = random_table(p0, [maxb * block] * B, 3)
    cache = sa.paged_cache(p0)
    codes, scale = [raw(c) for c in cache[:2]], [np.zeros((pages, Hkv)) for _ in "kv"]
    L = torch.full((B, Hkv, maxb, d), 7.0, dtype=T[dtype], device="cuda")
    Lref = np.full(L.shape, 7.0)
    for step, grown in enumerate(steps):
        lens = lens + np.array(grown)
        slot, cu = split_slots(p0, table, lens, grown, pad=4)
        n = len(slot)
        # later steps bring larger values to some tokens, so scales grow and codes are rounded anew
        x = [torch.from_numpy(rng.standard_normal((n, Hkv, d)) * rng.choice([0.01, 1.0, 9.0], (n, 1, 1)) * 3.0 ** step).to(T[dtype])
             for _ in "kv"]
        p = sa.make_paged_params(B, Hkv, Hkv, d, block, pages, maxb, n, code=code, dtype=dtype)
        ws = sa.paged_workspace(p)
        sa.paged_append(p, x[0].cuda(), x[1].cuda(), torch.tensor(slot, device="cuda"), cache, ws, cu=i32(cu),
                        new_len=i32(lens.tolist()), L=L)
        done(ws)
        for i in range(2):
            runs = op.append(CODE[code], block, x[i].double().numpy(), slot, codes[i], scale[i])
            assert np.array_equal(raw(cache[i]), codes[i]), (step, i)
            assert np.array_equal(cache[2 + i].double().cpu().numpy(), scale[i]), (step, i)
            for a, b_, page, off in runs if i == 0 else []:
                b = int(np.searchsorted(cu, a, side="right")) - 1
                held = off + b_ - a
                blk = int(np.where(table[b] == page)[0][0])
                Lref[b, :, blk] = op.values(CODE[code], codes[0][page:page + 1], scale[0][page:page + 1])[0, :, :held].mean(1)
        # one rounding to the type, and the sum of up to 128 codes and the division in fp32
        tol = (torch.finfo(T[dtype]).eps / 2 + 3 * 2.0 ** -24) * np.abs(Lref) + 2.0 ** -24 * (448 if code == "e4m3" else 127) * scale[0].max()
        assert (np.abs(L.double().cpu().numpy() - Lref) <= tol).all()
        # read back: every cached row, rounded once
        every, _ = split_slots(p, table, lens, lens, pad=2)
        pr = sa.make_paged_params(B, Hkv, Hkv, d, block, pages, maxb, len(every), code=code, dtype=dtype)
        got = sa.paged_gather(pr, torch.tensor(every, device="cuda"), cache, ws)
        done(ws)
        for i in range(2):
            vals = op.values(CODE[code], codes[i], scale[i])
            ref = np.stack([vals[s // block, :, s % block] if s >= 0 else np.zeros((Hkv, d)) for s in every])
            assert np.array_equal(got[i].double().cpu().numpy(), torch.from_numpy(ref).to(T[dtype]).double().numpy()), (step, i)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 64), ("bf16", 64, 128), ("fp32", 128, 80), ("bf16", 128, 16)])
def test_append_of_long_prompts(code, dtype, d, block):
    """Enough tokens that windows of several runs share a CTA, appended in two
    calls of ragged prompts and single tokens, some of them not finite."""
    rng = np.random.default_rng(block)
    B, Hkv = 130, 2
    grown = [[1] * B, [int(x) for x in rng.integers(0, 3, B)]]
    grown[0][5], grown[0][60] = 1500, 3 * block
    grown[1][5], grown[1][7], grown[1][61] = 2 * block + 5, 700, block - 1
    maxb = 2300 // block + 3
    lens = np.zeros(B, int)
    pages = sum(-(-(a + b) // block) for a, b in zip(*grown)) + 1
    p0 = sa.make_paged_params(B, Hkv, Hkv, d, block, pages, maxb, 0, code=code, dtype=dtype)
    table = random_table(p0, [a + b for a, b in zip(*grown)], 3)
    cache = sa.paged_cache(p0)
    codes, scale = [raw(c) for c in cache[:2]], [np.zeros((pages, Hkv)) for _ in "kv"]
    L = torch.zeros(B, Hkv, maxb, d, dtype=T[dtype], device="cuda")
    for step, g in enumerate(grown):
        lens = lens + np.array(g)
        slot, cu = split_slots(p0, table, lens, g, pad=2600)
        n = len(slot)
        x = [torch.from_numpy(rng.standard_normal((n, Hkv, d)) * 2.0 ** (step - 2)).to(T[dtype]) for _ in "kv"]
        x[0][7, 1, 3], x[1][200, 0, 0], x[1][201, 0, 1] = math.inf, math.nan, -math.inf
        p = sa.make_paged_params(B, Hkv, Hkv, d, block, pages, maxb, n, code=code, dtype=dtype)
        assert n * Hkv * 2 > 64 * 148          # one warp a token no longer
        ws = sa.paged_workspace(p, ops=[sa.SA_OP_PAGED_APPEND])
        sa.paged_append(p, x[0].cuda(), x[1].cuda(), torch.tensor(slot, device="cuda"), cache, ws, cu=i32(cu),
                        new_len=i32(lens.tolist()), L=L)
        torch.cuda.synchronize()
        assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 2)
        for i in range(2):
            op.append(CODE[code], block, x[i].double().numpy(), slot, codes[i], scale[i])
            assert np.array_equal(raw(cache[i]), codes[i]), (step, i)
            assert np.array_equal(cache[2 + i].double().cpu().numpy(), scale[i]), (step, i)
    vals = op.values(CODE[code], codes[0], scale[0])
    for b in (0, 5, 7, 60, 61, 129):
        for j in range(-(-int(lens[b]) // block)):
            ref = vals[table[b, j], :, :min(block, lens[b] - j * block)].mean(1)
            tol = (torch.finfo(T[dtype]).eps / 2 + 3 * 2.0 ** -24) * np.abs(ref) + 2.0 ** -24 * (448 if code == "e4m3" else 127) * scale[0].max()
            assert (np.abs(L[b, :, j].double().cpu().numpy() - ref) <= tol).all(), (b, j)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_append_of_what_is_not_finite(code):
    p = sa.make_paged_params(1, 1, 1, 64, 16, 2, 2, 3, code=code)
    cache, ws = sa.paged_cache(p), sa.paged_workspace(p)
    x = torch.randn(3, 1, 64, dtype=torch.float32).bfloat16()
    x[0, 0, 3], x[1, 0, 5], x[2, 0, 7] = math.nan, math.inf, -math.inf
    v = torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    slot = torch.tensor([16, 17, 18], device="cuda")
    sa.paged_append(p, x.cuda(), v.cuda(), slot, cache, ws)
    torch.cuda.synchronize()
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 2)
    codes, scale = np.zeros((2, 1, 16, 64), np.uint8), np.zeros((2, 1))
    op.append(CODE[code], 16, x.double().numpy(), [16, 17, 18], codes, scale)
    assert np.array_equal(raw(cache[0]), codes) and cache[2][1, 0].item() == scale[1, 0]
    assert not raw(cache[1]).any() and cache[3][1, 0].item() == 2.0 ** -126     # a block of zeros
    K, V = sa.paged_gather(p, slot, cache, ws)
    assert K[0, 0, 3] == 0 and K[1, 0, 5] == K.max() and torch.isfinite(K).all() and not V.any()


def test_append_skips_and_reports_bad_slots():
    p = sa.make_paged_params(1, 1, 1, 64, 16, 2, 2, 4)
    cache, ws = sa.paged_cache(p), sa.paged_workspace(p)
    x = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    sa.paged_append(p, x, x, torch.tensor([32, -1, 5, 1 << 40], device="cuda"), cache, ws)
    torch.cuda.synchronize()
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 1)
    got = raw(cache[0])
    assert got[0, 0, 5].all() and got.astype(bool).sum() == 64
    K, _ = sa.paged_gather(p, torch.tensor([32, -1, 5, 1 << 40], device="cuda"), cache, ws)
    torch.cuda.synchronize()
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 1)
    assert (K[2] == 1).all() and not K[0].any() and not K[1].any() and not K[3].any()


def test_rows_of_a_fused_projection_and_of_a_head_major_tensor():
    n, H, d = 37, 2, 128
    p = sa.make_paged_params(1, H, H, d, 16, 4, 4, n)
    ws, slot = sa.paged_workspace(p), torch.arange(n, device="cuda")
    fused = torch.randn(n, (4 + 2 * H) * d, device="cuda").bfloat16()
    K, V = (fused[:, i * d:(i + H) * d].view(n, H, d) for i in (4, 4 + H))
    a, b, c = sa.paged_cache(p), sa.paged_cache(p), sa.paged_cache(p)
    sa.paged_append(p, K, V, slot, a, ws)
    sa.paged_append(p, K.contiguous(), V.contiguous(), slot, b, ws)
    hm = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (K, V)]       # [H, n, d] in memory
    sa.paged_append(p, *hm, slot, c, ws)
    done(ws)
    for x, y, z in zip(a, b, c):
        assert np.array_equal(raw(x), raw(y)) and np.array_equal(raw(x), raw(z))
    out = tuple(torch.empty(H, n, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    sa.paged_gather(p, slot, a, ws, out=tuple(t.transpose(0, 1) for t in out))
    ref = sa.paged_gather(p, slot, a, ws)
    done(ws)
    assert all(torch.equal(x.transpose(0, 1), y) for x, y in zip(out, ref))


# ---- decode ------------------------------------------------------------------------

def spoil_tails(p, cache, table, lens):
    """Rows behind a sequence's last token hold whatever was there: NaN codes."""
    for b, n in enumerate(lens):
        if n % p.block:
            page = int(table[b, n // p.block])
            for c in cache[:2]:
                c.view(torch.uint8)[page, :, n % p.block:] = 0x7f


def lists_for(p, lens, seed):
    """Random kept blocks as a selection leaves them: sink, some, local."""
    rng = np.random.default_rng(seed)
    Hsel = p.Hq if p.flags & sa.SA_SELECT_PER_QHEAD else p.Hkv
    cap = p.top_k + 2
    idx = np.full((p.B, Hsel, cap), -1, np.int32)
    sc = np.zeros((p.B, Hsel, cap), np.float32)
    cnt = np.zeros((p.B, Hsel), np.int32)
    for b, n in enumerate(lens):
        nb = max(1, -(-n // p.block))
        for h in range(Hsel):
            mid = rng.permutation(np.arange(1, max(1, nb - 1)))[:int(rng.integers(0, p.top_k + 1))]
            keep = sorted({0, nb - 1} | {int(x) for x in mid})
            idx[b, h, :len(keep)], cnt[b, h] = keep, len(keep)
            sc[b, h, :len(keep)] = rng.standard_normal(len(keep)) * 2
    return idx, sc, cnt


def check_decode(p, dtype, lens, seed, lists=None, sample=None, ws=None):
    cache, codes, scale = random_cache(p, seed)
    table = random_table(p, lens, seed)
    spoil_tails(p, cache, table, lens)
    q = torch.from_numpy(np.random.default_rng(seed + 1).standard_normal((p.B, p.Hq, p.d))).to(T[dtype])
    ws = sa.paged_workspace(p) if ws is None else ws
    dl = None if lists is None else tuple(torch.from_numpy(x).cuda() for x in lists)
    o, lse = sa.paged_decode(p, q.cuda(), cache, i32(table.tolist()), i32(list(lens)), ws, lists=dl)
    done(ws)
    o2, lse2 = sa.paged_decode(p, q.cuda(), cache, i32(table.tolist()), i32(list(lens)), ws, lists=dl)
    done(ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    kv = [op.values(p.code, c, s) for c, s in zip(codes, scale)]
    qd = q.double().numpy() * (p.scale or p.d ** -0.5)
    G = p.Hq // p.Hkv
    for b, n in enumerate(lens):
        for h in range(p.Hq) if sample is None else sample:
            u = (b, h if p.flags & sa.SA_SELECT_PER_QHEAD else h // G)
            ref = op.decode_row(qd[b, h], kv[0], kv[1], table[b], n, h // G, p.block, p.flags,
                                *((lists[0][u], lists[1][u]) if lists else ()))
            check_row(dtype, o[b, h], lse[b, h], ref, n, p.d, (b, h, n))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,block,Hq,Hkv", [(128, 64, 8, 2), (64, 16, 5, 1), (128, 128, 16, 2), (64, 64, 24, 2),
                                            (128, 48, 3, 3), (128, 112, 40, 2), (64, 32, 16, 1)])
def test_decode_over_every_block(code, dtype, d, block, Hq, Hkv):
    lens = [0, 1, block, block + 1, 3 * block - 1, 700, 15]
    maxb = 700 // block + 2
    p = sa.make_paged_params(len(lens), Hq, Hkv, d, block, 8 * maxb, maxb, 0, code=code, dtype=dtype)
    check_decode(p, dtype, lens, Hq + d)


MODES = {"gate": sa.SA_SINK | sa.SA_LOCAL | sa.SA_GATE | sa.SA_CAUSAL, "plain": sa.SA_SINK | sa.SA_LOCAL,
         "hier": sa.SA_SINK | sa.SA_LOCAL | sa.SA_HIER,
         "perq": sa.SA_SINK | sa.SA_LOCAL | sa.SA_GATE | sa.SA_SELECT_PER_QHEAD}


@pytest.mark.parametrize("mode", sorted(MODES))
@pytest.mark.parametrize("code,dtype,d,block,Hq,Hkv,top_k", [
    ("e4m3", "bf16", 128, 64, 8, 2, 9), ("int8", "bf16", 128, 32, 12, 1, 5), ("e4m3", "fp32", 64, 16, 4, 2, 7),
    ("int8", "bf16", 64, 128, 6, 2, 0), ("e4m3", "bf16", 128, 16, 20, 1, 40)])
def test_decode_over_kept_blocks(mode, code, dtype, d, block, Hq, Hkv, top_k):
    lens = [900, 0, 1, block, 2 * block + 1, 333]
    maxb = 900 // block + 2
    p = sa.make_paged_params(len(lens), Hq, Hkv, d, block, 5 * maxb, maxb, 0, top_k, MODES[mode], dtype, code)
    check_decode(p, dtype, lens, top_k + block, lists=lists_for(p, lens, 5))


def test_decode_splits_long_sequences():
    """One long sequence beside short ones: its blocks are shared out."""
    lens = [20000, 3, 640, 9000]
    p = sa.make_paged_params(4, 8, 1, 128, 64, 480, 320, 0)
    check_decode(p, "bf16", lens, 4, sample=[0, 7])


def test_decode_lists_that_keep_nothing_and_bad_entries():
    p = sa.make_paged_params(2, 4, 1, 128, 64, 8, 4, 0, 3, MODES["plain"])
    cache, codes, scale = random_cache(p, 1)
    table, lens = random_table(p, [200, 200], 2), [200, 200]
    q = torch.randn(2, 4, 128, device="cuda").bfloat16()
    ws = sa.paged_workspace(p)
    idx = i32([[[-1, -1, -1, -1, -1]], [[0, 9, 3, -1, -1]]])
    sc, cnt = torch.zeros(2, 1, 5, device="cuda"), i32([[0], [3]])
    o, lse = sa.paged_decode(p, q, cache, i32(table.tolist()), i32(lens), ws, lists=(idx, sc, cnt))
    torch.cuda.synchronize()
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 1)
    assert not o[0].any() and torch.isneginf(lse[0]).all()
    kv = [op.values(p.code, c, s) for c, s in zip(codes, scale)]
    # entry 9 is skipped, and so is what follows it out of order
    for h in range(4):
        ref = op.decode_row(q[1, h].double().cpu().numpy() / 128 ** 0.5, kv[0], kv[1], table[1], 200, 0, 64, p.flags,
                            [0], [0.0])
        check_row("bf16", o[1, h], lse[1, h], ref, 200, 128, h)
    bad = table.copy()
    bad[1, 0] = 8
    o, lse = sa.paged_decode(p, q, cache, i32(bad.tolist()), i32(lens), ws, lists=(i32([[[0, 3, -1, -1, -1]]] * 2), sc, i32([[2], [2]])))
    torch.cuda.synchronize()
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 1)


def test_decode_magnitudes():
    """Large and tiny queries and scales, and a scale of zero, stay finite."""
    p = sa.make_paged_params(3, 8, 1, 128, 64, 12, 4, 0)
    cache, codes, scale = random_cache(p, 9)
    cache[2].mul_(1e-3)
    cache[3][3] = 0.0
    cache[3][4] = 1e20
    cache[3][5] = 1e-30
    q = torch.randn(3, 8, 128) * torch.tensor([1e3, 1e-30, 1e-3])[:, None, None]
    q[2, :, ::2] = 0
    q = q.bfloat16()
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    ws = sa.paged_workspace(p)
    o, lse = sa.paged_decode(p, q.cuda(), cache, i32(table.tolist()), i32([250, 256, 130]), ws)
    done(ws)
    ks, vs = cache[2].double().cpu().numpy(), cache[3].double().cpu().numpy()
    kv = [op.values(p.code, c, s) for c, s in zip(codes, (ks, vs))]
    for b, n in enumerate([250, 256, 130]):
        for h in range(8):
            ref = op.decode_row(q[b, h].double().numpy() / 128 ** 0.5, kv[0], kv[1], table[b], n, 0, 64, 0)
            check_row("bf16", o[b, h], lse[b, h], ref, n, 128, (b, h))


# ---- chunked prefill ------------------------------------------------------------------

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("code,dtype,d,block,Hq,Hkv", [
    ("e4m3", "bf16", 128, 64, 8, 2), ("int8", "bf16", 128, 32, 5, 1), ("e4m3", "bf16", 64, 128, 4, 4),
    ("int8", "bf16", 128, 48, 24, 2), ("e4m3", "bf16", 128, 16, 40, 1), ("int8", "fp32", 64, 64, 6, 2),
    ("int8", "bf16", 64, 64, 16, 2)])
def test_prefill_chunks(causal, code, dtype, d, block, Hq, Hkv):
    grown = [70, 0, 1, 257, 55, 3, 0]          # sequence 4: more queries than keys
    run_chunks(causal, code, dtype, d, block, Hq, Hkv, grown)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("code,d,block,Hq,Hkv,grown", [
    ("e4m3", 128, 64, 8, 2, [5, 0, 1, 9, 7, 3, 0]), ("int8", 128, 128, 4, 4, [12, 0, 1, 3, 2, 30, 0]),
    ("e4m3", 64, 16, 5, 1, [3, 0, 1, 2, 8, 1, 1]), ("int8", 64, 48, 24, 2, [1, 0, 1, 4, 1, 2, 0]),
    ("e4m3", 128, 112, 40, 1, [2, 0, 1, 1, 1, 1, 0]), ("int8", 128, 32, 4, 4, [1, 0, 1, 1, 1, 1, 1])])
def test_prefill_of_few_rows(causal, code, d, block, Hq, Hkv, grown):
    """Drafted tokens: few rows per list, some of them in one long run."""
    run_chunks(causal, code, "bf16", d, block, Hq, Hkv, grown)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("code,d,block,Hq,Hkv,grown", [
    ("e4m3", 128, 64, 8, 2, [150, 0, 1, 10, 11, 3, 0]), ("int8", 64, 16, 5, 1, [1, 0, 1, 8, 9, 200, 1]),
    ("int8", 128, 48, 24, 2, [3, 0, 1, 4, 2, 90, 4]), ("e4m3", 128, 112, 40, 1, [1, 0, 1, 2, 1, 1, 60]),
    ("e4m3", 64, 64, 132, 1, [9, 0, 1, 2, 1, 5, 0])])
def test_prefill_of_a_mixed_batch(causal, code, d, block, Hq, Hkv, grown):
    """Single tokens and drafts beside a prompt's chunk: sequences of up to 40
    rows a kv-head and of more are taken by different kernels."""
    run_chunks(causal, code, "bf16", d, block, Hq, Hkv, grown)


def run_chunks(causal, code, dtype, d, block, Hq, Hkv, grown):
    lens = [300, 0, 1, 257, 40, 600, 130]
    grown = list(grown)
    if grown[4] < 30:
        lens[4] = grown[4] - 1                 # more queries than keys
    if not causal:
        grown[1] = 2                           # queries of a sequence without keys
    maxb = 600 // block + 2
    cu = [0]
    for g in grown:
        cu.append(cu[-1] + g)
    p = sa.make_paged_params(len(lens), Hq, Hkv, d, block, 4 * maxb, maxb, cu[-1] + 9, 0, sa.SA_CAUSAL if causal else 0,
                             dtype, code)
    cache, codes, scale = random_cache(p, 3)
    table = random_table(p, lens, 3)
    spoil_tails(p, cache, table, lens)
    Q = torch.from_numpy(np.random.default_rng(1).standard_normal((p.tokens, Hq, d))).to(T[dtype])
    out = (torch.full((p.tokens, Hq, d), 5.0, dtype=T[dtype], device="cuda"), torch.full((p.tokens, Hq), 5.0, device="cuda"))
    ws = sa.paged_workspace(p)
    args = (p, Q.cuda(), i32(cu), cache, i32(table.tolist()), i32(lens), ws)
    O, lse = sa.paged_prefill(*args, out=out)
    done(ws)
    assert (O[cu[-1]:] == 5).all() and (lse[cu[-1]:] == 5).all()
    O2, lse2 = sa.paged_prefill(*args)
    done(ws)
    assert torch.equal(O[:cu[-1]], O2[:cu[-1]]) and torch.equal(lse[:cu[-1]], lse2[:cu[-1]])
    kv = [op.values(p.code, c, s) for c, s in zip(codes, scale)]
    for b, n in enumerate(lens):
        T_b = grown[b]
        for t in sorted({0, 1, T_b // 2, T_b - 1} & set(range(T_b))):
            see = max(0, n - T_b + t + 1) if causal else n
            for h in sorted({0, Hq // 2, Hq - 1}):
                ref = op.decode_row(Q[cu[b] + t, h].double().numpy() * d ** -0.5, kv[0], kv[1], table[b], see,
                                    h // (Hq // Hkv), block, 0)
                check_row(dtype, O[cu[b] + t, h], lse[cu[b] + t, h], ref, see, d, (b, t, h))


@pytest.mark.parametrize("tokens,dtype", [(12, "bf16"), (400, "bf16"), (12, "fp32")])
def test_prefill_refuses_offsets_that_overlap(tokens, dtype):
    p = sa.make_paged_params(4, 8, 2, 128, 64, 40, 8, tokens, flags=sa.SA_CAUSAL, dtype=dtype)
    cache, _, _ = random_cache(p, 8)
    lens = [400, 100, 64, 500]
    table = i32(random_table(p, lens, 8).tolist())
    q = torch.randn(tokens, 8, 128, device="cuda").to(T[dtype])
    ws = sa.paged_workspace(p)
    for cu in ([0, tokens, 0, tokens, 0], [0, 1, 2, 3, tokens + 1], [-1, 1, 2, 3, 4], [0, 3, 2, 3, 4]):
        out = (torch.full_like(q, 5.0), torch.full((tokens, 8), 5.0, device="cuda"))
        sa.paged_prefill(p, q, i32(cu), cache, table, i32(lens), ws, out=out)
        torch.cuda.synchronize()
        assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 1)
        assert (out[0] == 5).all() and (out[1] == 5).all()
    cu = i32([0, tokens // 2, tokens // 2, tokens, tokens])
    O, lse = sa.paged_prefill(p, q, cu, cache, table, i32(lens), ws)      # the next call is whole
    done(ws)
    assert torch.isfinite(O.float()).all() and torch.isfinite(lse).sum() > 0


@pytest.mark.parametrize("tokens,dtype", [(12, "bf16"), (400, "bf16"), (12, "fp32")])
def test_prefill_leaves_rows_before_the_first_sequence(tokens, dtype):
    p = sa.make_paged_params(2, 4, 1, 64, 32, 40, 8, tokens, flags=sa.SA_CAUSAL, dtype=dtype)
    cache, _, _ = random_cache(p, 8)
    table, lens, ws = i32(random_table(p, [250, 250], 8).tolist()), i32([250, 250]), sa.paged_workspace(p)
    q = torch.randn(tokens, 4, 64, device="cuda").to(T[dtype])
    out = (torch.full_like(q, 5.0), torch.full((tokens, 4), 5.0, device="cuda"))
    sa.paged_prefill(p, q, i32([3, 5, tokens - 2]), cache, table, lens, ws, out=out)
    done(ws)
    rows = torch.tensor([False] * 3 + [True] * (tokens - 5) + [False] * 2)
    for x in out:
        assert ((x.cpu() == 5).flatten(1).all(1) == ~rows).all()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("tokens,dtype,d,block", [(6, "bf16", 128, 64), (300, "bf16", 128, 64), (300, "bf16", 64, 16),
                                                  (300, "bf16", 128, 128), (6, "fp32", 64, 32)])
def test_attention_leaves_blocks_without_a_page_out(tokens, dtype, d, block, code):
    """Table entries out of range in the middle, at both ends and all over a sequence."""
    lens, maxb = [700, 700, 130, 260], -(-700 // block)
    p = sa.make_paged_params(4, 4, 2, d, block, 4 * maxb, maxb, tokens, 0, 0, dtype, code)
    cache, codes, scale = random_cache(p, 5)
    table = random_table(p, lens, 5)
    spoil_tails(p, cache, table, lens)
    bad = table.copy()
    last = -(-700 // block) - 1
    bad[0, [1, last - 1]] = [-1, p.pages]
    bad[1, [0, last]] = [-2 ** 31, 2 ** 31 - 1]
    bad[2, :-(-130 // block)] = -1
    cu = [0, tokens // 3, tokens // 2, tokens - 1, tokens]
    Q = torch.from_numpy(np.random.default_rng(1).standard_normal((tokens, 4, d))).to(T[dtype])
    ws = sa.paged_workspace(p)
    got = [sa.paged_prefill(p, Q.cuda(), i32(cu), cache, i32(bad.tolist()), i32(lens), ws)]
    torch.cuda.synchronize()
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 1)
    first = Q[cu[:4]].cuda()
    got.append(sa.paged_decode(p, first, cache, i32(bad.tolist()), i32(lens), ws))
    torch.cuda.synchronize()
    assert sa.sparse_attn_check_status(ws.data_ptr(), 0) == (sa.SA_ERR_DEVICE, 1)
    kv = [op.values(p.code, c, s) for c, s in zip(codes, scale)]
    for b, n in enumerate(lens):
        keep = [j for j in range(-(-n // block)) if 0 <= bad[b, j] < p.pages]
        for t in {0, cu[b + 1] - cu[b] - 1}:
            for h in (0, 3):
                ref = op.decode_row(Q[cu[b] + t, h].double().numpy() * d ** -0.5, kv[0], kv[1], table[b], n, h // 2, block, 0,
                                    keep, [0.0] * len(keep))
                check_row(dtype, got[0][0][cu[b] + t, h], got[0][1][cu[b] + t, h], ref, n, d, (b, t, h))
                if t == 0:
                    check_row(dtype, got[1][0][b, h], got[1][1][b, h], ref, n, d, (b, h))


def test_prefill_rows_are_decodes():
    """One query per sequence: the chunk call and the decode call agree."""
    lens = [5000, 64, 1]
    p = sa.make_paged_params(3, 8, 2, 128, 64, 100, 80, 3, flags=sa.SA_CAUSAL)
    cache, _, _ = random_cache(p, 8)
    table = i32(random_table(p, lens, 8).tolist())
    q = torch.randn(3, 8, 128, device="cuda").bfloat16()
    ws = sa.paged_workspace(p)
    o, lse = sa.paged_decode(p, q, cache, table, i32(lens), ws)
    O, lse2 = sa.paged_prefill(p, q, i32([0, 1, 2, 3]), cache, table, i32(lens), ws)
    done(ws)
    # two roundings of the weights and two of the output, on values of about 2
    assert (o.float() - O.float()).abs().max() <= 4 * 2.0 ** -8 * cache[0].float().abs().max() * 0.03 and \
        (lse - lse2).abs().max() <= 1e-4


# ---- together ---------------------------------------------------------------------------

def serve(steps, capture):
    """Prompts are cached, then every sequence decodes `steps` tokens through
    the selection's lists, all lengths and tables on the GPU."""
    torch.manual_seed(3)
    B, Hq, Hkv, d, bs, maxb, top_k = 3, 8, 2, 128, 64, 16, 3
    flags = sa.SA_SINK | sa.SA_LOCAL | sa.SA_GATE | sa.SA_CAUSAL
    prompts = [300, 17, 640]
    pages = 60
    dense = sa.make_params(B, Hq, Hkv, d, maxb * bs, bs, top_k, flags)
    dws = sa.workspace(dense, ops=sa.DECODE_OPS)
    free, n_free = torch.randperm(pages, device="cuda").int(), i32([pages])
    table = torch.full((B, maxb), -1, dtype=torch.int32, device="cuda")
    L = torch.zeros(B, Hkv, maxb, d, dtype=torch.bfloat16, device="cuda")
    cur, new = i32([0] * B), i32(prompts)
    pp = sa.make_paged_params(B, Hq, Hkv, d, bs, pages, maxb, 1000, top_k, flags)
    ps = sa.make_paged_params(B, Hq, Hkv, d, bs, pages, maxb, B, top_k, flags)
    cache = sa.paged_cache(pp)
    ws = sa.paged_workspace(pp)
    K, V = (torch.randn(1000, Hkv, d, device="cuda").bfloat16() for _ in "kv")
    nf, cu, slot = sa.paged_tables(pp, cur, new, free, n_free, table, ws)
    sa.paged_append(pp, K, V, slot, cache, ws, cu=cu, new_len=new, L=L)
    n_free.copy_(nf)
    cur.copy_(new)
    k1, v1 = (torch.randn(B, Hkv, d, device="cuda").bfloat16() for _ in "kv")
    q = torch.randn(B, Hq, d, device="cuda").bfloat16()
    outs = []

    def step():
        new.add_(1)
        nf, cu, slot = sa.paged_tables(ps, cur, new, free, n_free, table, ws)
        sa.paged_append(ps, k1, v1, slot, cache, ws, cu=cu, new_len=new, L=L)
        lists = sa.select_decode_varlen(dense, q, L, new, dws)
        o, lse = sa.paged_decode(ps, q, cache, table, new, ws, lists=lists)
        n_free.copy_(nf)
        cur.copy_(new)
        return o, lse, lists

    if capture:
        saved = [t.clone() for t in (new, n_free, cur, table, free, L, *cache)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        for t, s in zip((new, n_free, cur, table, free, L, *cache), saved):
            t.view(torch.uint8).copy_(s.view(torch.uint8))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse, lists = step()
        for t, s in zip((new, n_free, cur, table, free, L, *cache), saved):
            t.view(torch.uint8).copy_(s.view(torch.uint8))
        for i in range(steps):
            k1.add_(0.25)
            g.replay()
            outs.append((o.clone(), lse.clone(), lists[0].clone()))
    else:
        for i in range(steps):
            k1.add_(0.25)
            o, lse, lists = step()
            outs.append((o, lse, lists[0]))
    done(ws)
    done(dws)
    return outs, (B, Hkv, d, bs, maxb, pages, table, cache, new, q, lists, dense, dws, pp)


def test_a_serving_loop_and_its_capture():
    steps = 70                                  # past a block boundary for every sequence
    a, st = serve(steps, False)
    b, _ = serve(steps, True)
    for i, (x, y) in enumerate(zip(a, b)):
        assert all(torch.equal(s, t) for s, t in zip(x, y)), i
    # the last step against the framework's decode over the cache read back
    B, Hkv, d, bs, maxb, pages, table, cache, new, q, lists, dense, dws, pp = st
    pos = torch.arange(maxb * bs, device="cuda")
    slot = torch.where(pos < new[:, None], table.long()[:, pos // bs] * bs + pos % bs, -1)
    K, V = (torch.empty(B, Hkv, maxb * bs, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    pr = sa.make_paged_params(B, pp.Hq, Hkv, d, bs, pages, maxb, maxb * bs)
    ws = sa.paged_workspace(pr)
    for i in range(B):
        sa.paged_gather(pr, slot[i].contiguous(), cache, ws, out=(K[i].transpose(0, 1), V[i].transpose(0, 1)))
    o, lse = sa.decode_varlen(dense, q, K, V, new, *lists, dws)
    done(ws)
    # scales are powers of two, so the read-back is exact: two forms of one product, each with rounded weights
    assert (o.float() - a[-1][0].float()).abs().max() <= 4 * 2.0 ** -8 * V.float().abs().max()
    assert (lse - a[-1][1]).abs().max() <= 1e-3
    # landmarks: what the framework computes from the read-back keys
    Lr = torch.zeros(B, Hkv, maxb, d, dtype=torch.bfloat16, device="cuda")
    sa.landmarks_update(dense, K, Lr, seq_len=new)
    sel = sa.select_decode_varlen(dense, q, Lr, new, dws)
    done(dws)
    assert torch.equal(sel[0], lists[0])


def test_a_call_runs_on_the_stream_it_is_given():
    p = sa.make_paged_params(2, 8, 2, 128, 64, 20, 8, 0)
    cache, _, _ = random_cache(p, 2)
    table, n = i32(random_table(p, [500, 77], 2).tolist()), i32([500, 77])
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    ws = sa.paged_workspace(p)
    ref = sa.paged_decode(p, q, cache, table, n, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sa.paged_decode(p, q, cache, table, n, ws, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_a_cache_beyond_32_bit_offsets(code):
    """Codes of more than 4 GiB: the last pages are appended to, read back and
    attended to like the first ones."""
    block, H, d = 64, 2, 128
    pages = 4 * (1 << 30) // (block * H * d) + 300
    p = sa.make_paged_params(1, 8, H, d, block, pages, 16, 900, flags=sa.SA_CAUSAL, code=code)
    small = sa.make_paged_params(1, 8, H, d, block, 16, 16, 900, flags=sa.SA_CAUSAL, code=code)
    ct = torch.float8_e4m3fn if code == "e4m3" else torch.int8
    shape = (pages, H, block, d)
    big = tuple(torch.empty(shape, dtype=torch.uint8, device="cuda").view(ct) for _ in "kv") + tuple(
        torch.zeros(shape[:2], device="cuda") for _ in "kv")
    ref = sa.paged_cache(small)
    tables = [torch.arange(pages - 16, pages, device="cuda").int(), torch.arange(16, device="cuda").int()]
    K, V = (torch.randn(900, H, d, device="cuda").bfloat16() for _ in "kv")
    Q = torch.randn(900, 8, d, device="cuda").bfloat16()
    pos, cu, n = torch.arange(900, device="cuda"), i32([0, 900]), i32([900])
    got = []
    for q, cache, table in ((p, big, tables[0]), (small, ref, tables[1])):
        ws = sa.paged_workspace(q)
        slot = table.long()[pos // block] * block + pos % block
        sa.paged_append(q, K, V, slot, cache, ws)
        back = sa.paged_gather(q, slot, cache, ws)
        O, lse = sa.paged_prefill(q, Q, cu, cache, table, n, ws)
        one = sa.make_paged_params(1, 8, H, d, block, q.pages, 16, 3, flags=sa.SA_CAUSAL, code=code)
        o3, lse3 = sa.paged_prefill(one, Q[:3].contiguous(), i32([0, 3]), cache, table, n, ws)
        o, l1 = sa.paged_decode(q, Q[:1].contiguous(), cache, table, n, ws)
        done(ws)
        got.append((*back, O, lse, o3, lse3, o, l1))
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("tokens,grown", [(24, [9, 3]), (600, [333, 120])])
def test_prefill_captured_and_replayed(tokens, grown):
    p = sa.make_paged_params(2, 8, 2, 128, 64, 40, 16, tokens, flags=sa.SA_CAUSAL)
    cache, _, _ = random_cache(p, 2)
    lens = [700, 450]
    table, n, cu = i32(random_table(p, [1000, 1000], 2).tolist()), i32(lens), i32([0, grown[0], sum(grown)])
    Q = torch.randn(tokens, 8, 128, device="cuda").bfloat16()
    ws = sa.paged_workspace(p)
    sa.paged_prefill(p, Q, cu, cache, table, n, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        O, lse = sa.paged_prefill(p, Q, cu, cache, table, n, ws)
    for step in range(3):
        n.copy_(i32([700 + 97 * step, 450 - 64 * step]))
        cu.copy_(i32([0, grown[0] - step, sum(grown) - 2 * step]))
        Q.normal_()
        O.fill_(5)
        g.replay()
        ref, rl = sa.paged_prefill(p, Q, cu, cache, table, n, sa.paged_workspace(p))
        done(ws)
        m = sum(grown) - 2 * step
        assert torch.equal(O[:m], ref[:m]) and torch.equal(lse[:m], rl[:m]) and (O[m:] == 5).all()


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own."""
    p = sa.make_paged_params(4, 8, 2, 128, 64, 200, 40, 300, flags=sa.SA_CAUSAL)
    cache, _, _ = random_cache(p, 2)
    lens = [2500, 77, 1, 1300]
    table, n, cu = i32(random_table(p, lens, 2).tolist()), i32(lens), i32([0, 200, 201, 202, 300])
    q, Q = torch.randn(4, 8, 128, device="cuda").bfloat16(), torch.randn(300, 8, 128, device="cuda").bfloat16()
    ref = (*sa.paged_decode(p, q, cache, table, n, sa.paged_workspace(p)),
           *sa.paged_prefill(p, Q, cu, cache, table, n, sa.paged_workspace(p)))
    ws, streams = [sa.paged_workspace(p) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(streams[0]):
            a = sa.paged_decode(p, q, cache, table, n, ws[0])
        with torch.cuda.stream(streams[1]):
            b = sa.paged_prefill(p, Q, cu, cache, table, n, ws[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ref, (*a, *b)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_query_that_is_not_a_number_spoils_its_own_row(dtype):
    p = sa.make_paged_params(3, 8, 2, 128, 64, 40, 16, 300, flags=sa.SA_CAUSAL, dtype=dtype)
    cache, _, _ = random_cache(p, 2)
    table, n, cu = i32(random_table(p, [500] * 3, 2).tolist()), i32([500, 321, 64]), i32([0, 150, 299, 300])
    Q = torch.randn(300, 8, 128, device="cuda").to(T[dtype])
    ws = sa.paged_workspace(p)
    O, lse = sa.paged_prefill(p, Q, cu, cache, table, n, ws)
    o, l1 = sa.paged_decode(p, Q[:3].contiguous(), cache, table, n, ws)
    bad = Q.clone()
    bad[1, 3, 7], bad[200, 0, 0] = math.nan, math.inf
    O2, lse2 = sa.paged_prefill(p, bad, cu, cache, table, n, ws)
    o2, l2 = sa.paged_decode(p, bad[:3].contiguous(), cache, table, n, ws)
    done(ws)
    keep = torch.ones(300, 8, dtype=torch.bool, device="cuda")
    keep[1, 3] = keep[200, 0] = False
    assert torch.equal(O[keep], O2[keep]) and torch.equal(lse[keep], lse2[keep]) and torch.isnan(O2[1, 3].float()).all()
    assert torch.equal(o[keep[:3]], o2[keep[:3]]) and torch.equal(l1[keep[:3]], l2[keep[:3]]) and torch.isnan(o2[1, 3].float()).all()
