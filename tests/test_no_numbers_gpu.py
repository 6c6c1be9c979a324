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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_every_scale(sd, dim, dtype):
    """One key a lane.  The output is its value, lse its score: codes times 2^(scale - 127), in fp16 2^-14 at least."""
    import torch
    scales, ps = list(range(135)), 16
    lanes = len(scales)
    codes = [c for c in range(256) if c & 127 != 127]
    codes = [codes[i * 3 % len(codes)] for i in range(dim)]
    size = 2.0 ** np.maximum(np.array(scales, np.float64) - 127, -14.0 if dtype == "f16" else -127.0)
    v, k = np.zeros((lanes, ps, 1, dim), np.uint8), np.zeros((lanes, ps, 1, dim), np.uint8)
    v[:, 0, 0], k[:, 0, 0, 0] = codes, 0x38
    ks, vs = np.full((lanes, 1, ps), 127, np.uint8), np.full((lanes, 1, ps), 127, np.uint8)
    t = lambda x: torch.tensor(x, device="cuda")  # noqa: E731
    q = torch.zeros((lanes, 2, dim), dtype=_dt(dtype), device="cuda")
    q[:, 0, 0], q[:, 1, 0] = 1.0, -0.5
    b = _batch(sd, [[i] for i in range(lanes)], list(range(lanes + 1)), [1] * lanes, ps)
    tiny = torch.finfo(_dt(dtype)).tiny
    # the values' scales: exact, but for what the tensor cores and the output's type have below the smallest normal number
    vs[:, 0, 0] = scales
    out, lse = _attend(sd, q, sd.PagedCache8(t(k), t(ks), t(v), t(vs), dtype=_dt(dtype)), b, None, 1.0, 0, 1, True)
    want = torch.tensor(ref.code_values()[codes] * size[:, None])
    for h in range(2):
        off = (out[:, h].cpu().double() - want).abs()
        assert off[want.abs() >= tiny].max() == 0 and off.max() < tiny
    # exponents of up to 2^7 in size and of 7 less, rounded: 2^-18 each
    assert (lse - torch.tensor([1.0, -0.5], device="cuda")).abs().max() <= 2.0 ** -17
    # the keys'
    ks[:, 0, 0], vs[:, 0, 0] = scales, 127
    out, lse = _attend(sd, q, sd.PagedCache8(t(k), t(ks), t(v), t(vs), dtype=_dt(dtype)), b, None, 1.0, 0, 1, True)
    for h, x in enumerate((1.0, -0.5)):
        assert (lse[:, h].cpu().double() - torch.tensor(size * x)).abs().max() <= 2.0 ** -20 * 128
        at = [i for i, s in enumerate(size) if s >= 2.0 ** -14]
        assert ((lse[at, h].cpu().double() - torch.tensor(size[at] * x)).abs() <= 2.0 ** -20 * torch.tensor(size[at]).clamp(min=8.0)).all()


def test_smallest_scales_of_both(sd):
    """Keys and values of bf16 caches with scales below those that the store writes: a key times 2^100 in q tells 2^-127 from
    2^-120."""
    import torch
    ps = 16
    for dim in (64, 128, 256):
        for byte in range(8):
            k = torch.zeros((1, ps, 1, dim), dtype=torch.uint8, device="cuda")
            k[0, :2, 0, 0] = 0x38
            ks = torch.full((1, 1, ps), 127, dtype=torch.uint8, device="cuda")
            ks[0, 0, 0], ks[0, 0, 1] = byte, 0
            cache = sd.PagedCache8(k, ks, torch.zeros_like(k), ks.clone(), dtype=torch.bfloat16)
            q = torch.zeros((1, 1, dim), dtype=torch.bfloat16, device="cuda")
            q[0, 0, 0] = 2.0 ** 125
            _, lse = _attend(sd, q, cache, _batch(sd, [[0]], [0, 1], [2], ps), None, 1.0, 0, 1, True)
            want = np.logaddexp(2.0 ** (byte - 2), 2.0 ** -2)
            assert abs(float(lse) - want) <= 2.0 ** -16 * max(1.0, want), (dim, byte, float(lse), want)
