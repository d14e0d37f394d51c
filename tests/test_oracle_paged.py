"""The paged cache's oracle against torch's own conversions and dense attention,
and the host-side refusals of the paged entry points (no GPU)."""
import numpy as np
import pytest
import torch

import block_sparse_long_landmark_b200 as sa
from block_sparse_long_landmark_b200 import build as sabuild
from oracle import paged as op


def test_e4m3_codes_are_torchs():
    raw = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(raw).view(torch.float8_e4m3fn).double().numpy()
    assert np.isnan(ref).sum() == 2 and np.array_equal(op.decode_codes(op.E4M3, raw), ref, equal_nan=True)


@pytest.mark.parametrize("seed", range(3))
def test_e4m3_rounding_is_torchs(seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(20000, generator=g) * 2.0 ** torch.randint(-12, 8, (20000,), generator=g)
    x = torch.cat([x.clamp(-448, 448), torch.arange(0, 512) / 1024.0, torch.arange(0, 448) + 0.5])
    ref = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(op.encode(op.E4M3, x.double().numpy()), ref)


def test_int8_rounding_is_torchs():
    x = torch.cat([torch.randn(5000) * 40, torch.arange(-300, 300) / 2])
    ref = x.round().clamp(-127, 127).to(torch.int8).numpy().view(np.uint8)
    assert np.array_equal(op.encode(op.INT8, x.double().numpy()), ref)


@pytest.mark.parametrize("code", [op.E4M3, op.INT8])
def test_scale_is_the_smallest_power_of_two(code):
    M = op.MOST[code]
    for amax in [1e-30, M * 0.5, np.nextafter(M, 0), M, np.nextafter(M, 1e9), 3.0, 1e30]:
        s = op.scale_for(code, amax)
        assert amax <= M * s and (amax > M * s / 2 or s == 2.0 ** -126)
    assert op.scale_for(code, 0.0) == 2.0 ** -126


def test_tables_pop_what_was_pushed_last():
    table = np.full((3, 4), -1)
    table[0, :2] = [7, 3]
    # sequence 0 ends (pages 7, 3 back), sequence 1 takes two pages, sequence 2 one
    n, t, free, cu, slot = op.tables([20, 0, 0], [0, 17, 1], [5, 6, 0, 0, 0, 0, 0, 0], 2, table, 16, 20)
    assert list(t[1, :2]) == [3, 7] and t[2, 0] == 6 and n == 1 and free[0] == 5 and cu == [0, 0, 17, 18]
    assert slot[0] == 48 and slot[16] == 112 and slot[17] == 96 and slot[18:] == [-1, -1]
    assert op.tables([0], [100], [1, 2, 3], 3, np.full((1, 8), -1), 16, 200) is None
    assert op.tables([0], [10], [1, 2, 3], 3, np.full((1, 8), -1), 16, 9) is None


@pytest.mark.parametrize("code", [op.E4M3, op.INT8])
def test_append_in_steps_keeps_the_largest_value(code):
    rng = np.random.default_rng(0)
    codes, scale = np.zeros((3, 2, 16, 64), np.uint8), np.zeros((3, 2))
    x = rng.standard_normal((12, 2, 64))
    x[9] *= 50
    op.append(code, 16, x[:5], [16, 17, 18, 19, 20], codes, scale)
    op.append(code, 16, x[5:], [21 + i for i in range(7)], codes, scale)
    v = op.values(code, codes, scale)[1, :, :12].transpose(1, 0, 2)
    step = scale[1].max() * (32 if code == op.E4M3 else 1)
    assert np.abs(v - x).max() <= step and not codes[0].any() and not codes[2].any()


def test_attention_is_dense_attention():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 120, (4, 1, 16, 64)).astype(np.uint8)
    scale = rng.random((4, 1)) * 0.01
    vals = op.values(op.E4M3, codes, scale)
    q = rng.standard_normal(64) / 8
    o, lse, _, _ = op.decode_row(q, vals, vals, [2, 0, 3], 37, 0, 16, 0)
    k = torch.from_numpy(np.concatenate([vals[2, 0], vals[0, 0], vals[3, 0]])[:37])
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q)[None, None], k[None], k[None], scale=1.0)
    assert np.abs(o - ref[0, 0].numpy()).max() < 1e-12
    assert abs(lse - float(torch.logsumexp(k @ torch.from_numpy(q), 0))) < 1e-12


# ---- refusals: every check fails before a launch ---------------------------

A = 256      # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    sabuild.build()


def _p(**kw):
    base = dict(B=2, Hq=8, Hkv=2, d=128, block=64, pages=32, max_blocks=8, tokens=10, top_k=4, flags=0)
    base.update(kw)
    return sa.make_paged_params(**base)


def _calls(p, n=1 << 40):
    return {
        "tables": sa.sparse_attn_paged_tables(p, A, A, A, A, 2 * A, A, A, A, A, n, None),
        "append": sa.sparse_attn_paged_append(p, A, A, 0, 0, A, None, None, A, A, A, A, None, A, n, None),
        "gather": sa.sparse_attn_paged_gather(p, A, A, A, A, A, A, A, 0, 0, A, n, None),
        "decode": sa.sparse_attn_paged_decode(p, A, A, A, A, A, A, A, None, None, None, A, A, A, n, None),
        "prefill": sa.sparse_attn_paged_prefill(p, A, A, A, A, A, A, A, A, A, A, A, n, None),
    }


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), sa.SA_ERR_ARG), (dict(Hq=7), sa.SA_ERR_ARG), (dict(pages=0), sa.SA_ERR_ARG),
    (dict(max_blocks=0), sa.SA_ERR_ARG), (dict(tokens=-1), sa.SA_ERR_ARG), (dict(top_k=257), sa.SA_ERR_ARG),
    (dict(flags=64), sa.SA_ERR_ARG), (dict(dtype=5), sa.SA_ERR_ARG), (dict(code=2), sa.SA_ERR_ARG),
    (dict(scale=-1.0), sa.SA_ERR_ARG), (dict(scale=float("nan")), sa.SA_ERR_ARG),
    (dict(d=96), sa.SA_ERR_UNSUPPORTED), (dict(block=24), sa.SA_ERR_UNSUPPORTED), (dict(block=144), sa.SA_ERR_UNSUPPORTED),
    (dict(B=16385), sa.SA_ERR_UNSUPPORTED), (dict(pages=1 << 24), sa.SA_ERR_UNSUPPORTED),
    (dict(max_blocks=1 << 25), sa.SA_ERR_UNSUPPORTED),
    (dict(flags=sa.SA_GATE), sa.SA_ERR_UNSUPPORTED),
    (dict(flags=sa.SA_GATE | sa.SA_LOCAL | sa.SA_HIER), sa.SA_ERR_UNSUPPORTED),
])
def test_bad_parameters_are_refused(kw, code):
    p = _p(**kw)
    assert _calls(p) == dict.fromkeys(("tables", "append", "gather", "decode", "prefill"), code)
    assert all(sa.sparse_attn_paged_workspace_size(p, op_) == 0 for op_ in range(5))


def test_small_workspaces_are_refused():
    p = _p()
    assert _calls(p, 16) == dict.fromkeys(("tables", "append", "gather", "decode", "prefill"), sa.SA_ERR_WORKSPACE)
    for op_ in range(5):
        assert sa.sparse_attn_paged_workspace_size(p, op_) >= 256
    assert sa.sparse_attn_paged_workspace_size(p, 9) == 0


def test_missing_and_misaligned_pointers_are_refused():
    p, n = _p(), 1 << 40
    good = [A, A, A, A, 2 * A, A, A, A, A]
    for i in range(9):
        bad = list(good)
        bad[i] = None
        assert sa.sparse_attn_paged_tables(p, *bad, n, None) == sa.SA_ERR_ARG, i
    assert sa.sparse_attn_paged_tables(p, A, A, A, A, A, A, A, A, A, n, None) == sa.SA_ERR_ARG   # n_free in place
    # K V slot K8 V8 kscale vscale ws
    def app(K=A, V=A, ts=0, hs=0, slot=A, cu=None, nl=None, K8=A, V8=A, ks=A, vs=A, L=None, ws=A, p=p):
        return sa.sparse_attn_paged_append(p, K, V, ts, hs, slot, cu, nl, K8, V8, ks, vs, L, ws, n, None)
    for kw in (dict(K=None), dict(V=None), dict(slot=None), dict(K8=None), dict(V8=None), dict(ks=None), dict(vs=None),
               dict(ws=None), dict(K=A + 8), dict(K8=A + 8), dict(L=A), dict(L=A, cu=A), dict(L=A + 8, cu=A, nl=A),
               dict(ts=256, hs=0), dict(ts=260, hs=128), dict(ts=128, hs=128), dict(ts=64, hs=1280)):
        assert app(**kw) == sa.SA_ERR_ARG, kw
    def gat(slot=A, K8=A, K=A, V=A, ts=0, hs=0, ws=A):
        return sa.sparse_attn_paged_gather(p, slot, K8, A, A, A, K, V, ts, hs, ws, n, None)
    for kw in (dict(slot=None), dict(K8=None), dict(K=None), dict(V=A + 2), dict(ws=None), dict(ts=8, hs=8)):
        assert gat(**kw) == sa.SA_ERR_ARG, kw
    good = [A] * 7 + [A, A, A] + [A, A, A]        # q K8 V8 ks vs table len | idx score count | o lse ws
    for i in range(13):
        bad = list(good)
        bad[i] = None
        assert sa.sparse_attn_paged_decode(p, *bad, n, None) == sa.SA_ERR_ARG, i
    for fl in (sa.SA_GATE | sa.SA_LOCAL, sa.SA_HIER):
        q = _p(flags=fl)
        assert sa.sparse_attn_paged_decode(q, *[A] * 7, None, None, None, A, A, A, n, None) == sa.SA_ERR_UNSUPPORTED
        assert sa.sparse_attn_paged_prefill(q, *[A] * 11, n, None) == sa.SA_ERR_UNSUPPORTED
    for i in range(11):
        bad = [A] * 11
        bad[i] = None
        assert sa.sparse_attn_paged_prefill(p, *bad, n, None) == sa.SA_ERR_ARG, i


def test_the_binding_refuses_other_tensors():
    p = _p(tokens=4, Hkv=2)
    cache = sa.paged_cache(p, device="cpu")
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    K = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    slot = torch.zeros(4, dtype=torch.int64)
    table, n = torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    for call in (
        lambda: sa.paged_append(p, K.float(), K.float(), slot, cache, ws),
        lambda: sa.paged_append(p, K[:3], K[:3], slot, cache, ws),
        lambda: sa.paged_append(p, K, K.transpose(0, 1).contiguous().transpose(0, 1), slot, cache, ws),
        lambda: sa.paged_append(p, K, K, slot.int(), cache, ws),
        lambda: sa.paged_append(p, K, K, slot, cache, ws, L=K),
        lambda: sa.paged_gather(p, slot[:2], cache, ws),
        lambda: sa.paged_decode(p, q[:, ::2], cache, table, n, ws),
        lambda: sa.paged_decode(p, q, (cache[0].view(torch.int8),) + cache[1:], table, n, ws),
        lambda: sa.paged_decode(p, q, cache, table.long(), n, ws),
        lambda: sa.paged_prefill(p, q, n, cache, table, n, ws),
        lambda: sa.paged_tables(p, n, n, n, n, table, ws),
        lambda: sa.paged_gather(p, slot, cache, ws),                   # all in order, but not on a GPU
        lambda: sa.paged_decode(p, q, cache, table, n, ws),
    ):
        with pytest.raises(sa.SparseAttnError) as e:
            call()
        assert e.value.code == sa.SA_ERR_ARG


def test_the_binding_refuses_expanded_rows():
    """Strides of 0 and 0 mean dense rows to the library: never an expanded tensor's."""
    p, one = _p(tokens=4, Hkv=2), _p(tokens=1, Hkv=2)
    ws, x = torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    for q in (p, one):
        cache, slot, rows = sa.paged_cache(q, device="cpu"), torch.zeros(q.tokens, dtype=torch.int64), x.expand(q.tokens, 2, 128)
        for call in (lambda: sa.paged_append(q, rows, rows, slot, cache, ws),
                     lambda: sa.paged_gather(q, slot, cache, ws, out=(rows, rows))):
            with pytest.raises(sa.SparseAttnError, match="expanded"):
                call()
