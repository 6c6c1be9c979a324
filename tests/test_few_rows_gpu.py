"""Few rows a key/value head over the 8-bit cache (heads of 128): the form with transposed products, against the plain
float64 form.  Needs a GPU."""
from __future__ import annotations

import numpy as np
import pytest

from tests import tree_ref as ref
from tests.test_tree_gpu import _attend, _batch, _cache, _check, _cu, _dt, _step

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


CASES = [
    # sizes, cached, kv heads, group, page, dtype, window, max_new (1 takes this form whatever the lanes have)
    ([1], [0], 1, 1, 16, "bf16", 0, 1), ([1], [127], 1, 16, 16, "f16", 0, 1), ([1] * 5, [0, 1, 128, 3_000, 255], 2, 5, 32, "bf16", 0, 1),
    ([16], [200], 1, 1, 64, "bf16", 0, 16), ([4, 2], [90, 5_000], 2, 4, 128, "f16", 0, 4),
    ([30, 0, 1, 9], [70, 5, 1_000, 0], 2, 4, 16, "bf16", 0, 1),          # lanes of many more rows than expected: many items
    ([2, 3], [4_000, 300], 1, 4, 16, "bf16", 256, 1), ([40], [600], 1, 3, 32, "f16", 100, 1),
    ([1], [12_000], 1, 4, 64, "bf16", 0, 1),                             # parts of one item in many CTAs
    ([1] * 24, list(range(0, 2_400, 100)), 2, 4, 64, "bf16", 0, 1),
]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_few_rows(sd, case, tree):
    import torch
    sizes, ctx, hk, group, ps, dtype, window, max_new = case
    if tree and 0 < window < 256:
        pytest.skip("a tree's window is 256 at least")
    rng = np.random.default_rng(sum(sizes) + group)
    seq, table, k, v, q = _step(sizes, ctx, hk, group, 128, ps, dtype, seed=group + len(sizes), window=window)
    # rows of different sizes, so that their factors differ
    q = (q.double() * torch.tensor(2.0 ** rng.integers(-4, 4, (q.shape[0], q.shape[1], 1)), device="cuda")).to(q.dtype)
    cache, (kk, vv) = _cache(sd, k, v, dtype, True)
    cu = _cu(sizes)
    masks = rng.integers(0, 1 << 32, (cu[-1], 2), dtype=np.uint64).astype(np.uint32) if tree else None
    want = ref.attention(q.double().cpu().numpy(), kk, vv, table, cu, seq, masks, 128 ** -0.5, window, dtype)
    m = torch.tensor(masks.view(np.int32), device="cuda") if tree else None
    got, lse = _attend(sd, q, cache, _batch(sd, table.tolist(), cu, seq, ps), m, 128 ** -0.5, window, max_new, True)
    _check(got, lse, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["large first", "zeros first", "in turn"])
def test_values_of_extreme_scales(sd, dtype, order):
    """Scores alike; half the keys' values with the largest scale, half zeros with the least (in one tile, or in one
    before the other): zeros weigh as much as the rest.  The scores are 0, so the sums are exact: the output is half the mean of the
    large values, which are one power of two."""
    import torch
    n, ps, dim = 512, 16, 128
    least = ref.least(dtype) + 127
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    k, v = z(n // ps, ps, 1, dim), z(n // ps, ps, 1, dim)
    ks, vs = z(n // ps, 1, ps) + 127, z(n // ps, 1, ps) + least
    i = torch.arange(n, device="cuda")
    big = {"large first": i < n // 2, "zeros first": i >= n // 2, "in turn": i % 2 == 0}[order].view(n // ps, ps)
    v[big] = 0x38                                             # 1
    vs[:, 0][big] = 134 if dtype == "bf16" else 130           # 2^7, 2^3
    cache = sd.PagedCache8(k, ks, v, vs, dtype=_dt(dtype))
    b = _batch(sd, [list(range(n // ps))], [0, 1], [n], ps)
    q = torch.ones((1, 3, dim), dtype=_dt(dtype), device="cuda")
    out, lse = _attend(sd, q, cache, b, None, 0.1, 0, 1, True)
    assert (out.float() == (64.0 if dtype == "bf16" else 4.0)).all()
    assert (lse - np.log(n)).abs().max() <= 2.0 ** -20 * np.log(n)


def test_rows_of_no_numbers(sd):
    """A row of q with a NaN, or an infinity, gives no numbers; the others are as without it."""
    import torch
    seq, table, k, v, q = _step([1, 1], [300, 20], 1, 6, 128, 16, "bf16", seed=2)
    cache, _ = _cache(sd, k, v, "bf16", True)
    b = _batch(sd, table.tolist(), [0, 1, 2], seq, 16)
    good, _ = _attend(sd, q, cache, b, None, 0.1, 0, 1, True)
    bad = q.clone()
    bad[0, 2, 5] = float("nan")
    got, _ = _attend(sd, bad, cache, b, None, 0.1, 0, 1, True)
    assert torch.isnan(got[0, 2]).all()
    got[0, 2] = good[0, 2]
    assert torch.equal(got, good)
