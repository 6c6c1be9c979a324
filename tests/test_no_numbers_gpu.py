"""Scales of the 8-bit cache that stand for no number, and the smallest ones, in every form of the attention: one answer
whatever the head size, the type and the number of rows.  Needs a GPU."""
from __future__ import annotations

import numpy as np
import pytest

from tests import tree_ref as ref
from tests.test_tree_gpu import _attend, _batch, _cache, _dt, _step

pytestmark = pytest.mark.gpu

# new tokens, query heads a key/value head, max_new: at most 16 rows (heads of 128 have a form of their own), one row tile, two
ROWS = [(4, 2, 1), (20, 2, 20), (70, 2, 70)]


@pytest.fixture(scope="module")
def sd():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g._load_build_module().build()
    import speculative_decoding_draft_column_gb300 as sd
    return sd


@pytest.mark.parametrize("scale", [135, 200, 254, 255])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scales_of_no_number(sd, dim, dtype, rows, scale):
    """Above 134, whatever the codes are: a key's makes the rows that see it NaN, a value's their outputs."""
    import torch
    (n, group, max_new), ctx, ps = rows, 30, 16
    seq, table, k, v, q = _step([n], [ctx], 1, group, dim, ps, dtype, seed=n + dim)
    cache, _ = _cache(sd, k, v, dtype, True)
    b = _batch(sd, table.tolist(), [0, n], seq, ps)
    good, lse = _attend(sd, q, cache, b, None, 0.125, 0, max_new, True)

    def at(j):
        return int(table[0][j // ps]), 0, j % ps

    kept = int(cache.k_scales[at(ctx + 2)])
    cache.k_scales[at(ctx + 2)] = scale
    out, _ = _attend(sd, q, cache, b, None, 0.125, 0, max_new, True)
    nan = torch.isnan(out).flatten(1)
    assert not nan[:2].any() and nan[2:].all() and torch.equal(out[:2], good[:2])
    cache.k_scales[at(ctx + 2)] = kept
    for codes in (None, 0):                              # a value that all rows see
        kept, codes_kept = int(cache.v_scales[at(3)]), cache.v[at(3)[0], at(3)[2], 0].clone()
        cache.v_scales[at(3)] = scale
        if codes is not None:
            cache.v[at(3)[0], at(3)[2], 0] = codes
        out, again = _attend(sd, q, cache, b, None, 0.125, 0, max_new, True)
        cache.v_scales[at(3)], cache.v[at(3)[0], at(3)[2], 0] = kept, codes_kept
        assert torch.isnan(out).all()
        # (at most 16 rows of 128: the value's scale takes part in the scores)
        assert torch.equal(again, lse) if dim != 128 or max_new > 1 else torch.isnan(again).all()
    # past the lane's last position it does not matter
    if (ctx + n) % ps:
        cache.v_scales[at(ctx + n)] = cache.k_scales[at(ctx + n)] = scale
    out, again = _attend(sd, q, cache, b, None, 0.125, 0, max_new, True)
    assert torch.equal(out, good) and torch.equal(again, lse)
