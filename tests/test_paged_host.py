"""Host-side sizes of the paged entry points (no GPU): what a workspace is
sized by."""
import pytest

import block_sparse_long_landmark_b200 as sa
from block_sparse_long_landmark_b200 import build as sabuild


@pytest.fixture(scope="module", autouse=True)
def built():
    sabuild.build()


def _size(op, **kw):
    base = dict(B=4, Hq=32, Hkv=2, d=128, block=64, pages=64, max_blocks=8, tokens=0)
    base.update(kw)
    return sa.sparse_attn_paged_workspace_size(sa.make_paged_params(**base), op)


@pytest.mark.parametrize("Hq,Hkv", [(32, 2), (32, 8), (40, 1), (6, 6)])
def test_a_decode_with_lists_per_query_head_has_room_for_one_without_lists(Hq, Hkv):
    f = sa.SA_SELECT_PER_QHEAD
    assert _size(sa.SA_OP_PAGED_DECODE, Hq=Hq, Hkv=Hkv, flags=f) >= _size(sa.SA_OP_PAGED_DECODE, Hq=Hq, Hkv=Hkv)


@pytest.mark.parametrize("B,tokens", [(1, 9), (1, 30), (2, 64), (8, 40), (64, 256), (64, 257), (300, 4000), (2, 0)])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (8, 8), (264, 2)])
def test_a_chunk_calls_workspace_is_not_sized_by_the_tables(B, tokens, Hq, Hkv):
    """Which kernels a call runs depends on the tables' length, what it needs does not."""
    kw = dict(B=B, tokens=tokens, Hq=Hq, Hkv=Hkv)
    sizes = {_size(sa.SA_OP_PAGED_PREFILL, max_blocks=m, pages=n, block=b, **kw)
             for m, n, b in ((1, 1, 16), (8, 64, 64), (2048, 64, 64), (1 << 16, 1 << 14, 128))}
    assert len(sizes) == 1 and min(sizes) >= 256
