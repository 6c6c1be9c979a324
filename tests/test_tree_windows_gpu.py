"""Trees with a window, over masks of any bits: a row whose mask is empty stands at the context, and sees the cached keys above
context - window.  Needs a GPU."""
from __future__ import annotations

import numpy as np
import pytest

from tests import tree_ref as ref
from tests.test_tree_gpu import _attend, _batch, _cache, _check, _step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sd():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g._load_build_module().build()
    import speculative_decoding_draft_column_gb300 as sd
    return sd


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("n,dim,group,max_new", [(40, 64, 2, 40), (40, 128, 4, 40), (40, 256, 1, 40), (7, 128, 2, 7)])
def test_empty_masks_and_a_window(sd, n, dim, group, max_new, eight):
    import torch
    rng = np.random.default_rng(n + dim)
    ctx, window, ps = 700, 256, 16
    seq, table, k, v, q = _step([n], [ctx], 1, group, dim, ps, "bf16", seed=dim, window=window)
    cache, (kk, vv) = _cache(sd, k, v, "bf16", eight)     # (before the window the cache holds anything)
    masks = rng.integers(0, 1 << 32, (n, 2), dtype=np.uint64).astype(np.uint32)
    masks[::3] = 0
    masks[5] = [~np.uint32((2 << 5) - 1), 0xFFFFFFFF]     # only bits above node 5
    lo = [ref.seen_keys(masks[i], ctx, i, window)[0] for i in (0, 3, 5)]
    assert lo == [ctx - window + 1] * 3
    want = ref.attention(q.double().cpu().numpy(), kk, vv, table, [0, n], seq, masks, dim ** -0.5, window, "bf16")
    b = _batch(sd, table.tolist(), [0, n], seq, ps)
    got, lse = _attend(sd, q, cache, b, torch.tensor(masks.view(np.int32), device="cuda"), dim ** -0.5, window, max_new, eight)
    _check(got, lse, want)
