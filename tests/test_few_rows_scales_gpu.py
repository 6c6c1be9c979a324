"""Few rows a key/value head over the 8-bit cache (heads of 128): values whose scales lie far apart, with scores that differ.
A key counts in the sum by its score alone, whatever its value's scale is.  Needs a GPU."""
from __future__ import annotations

import math

import numpy as np
import pytest

from tests import tree_ref as ref
from tests.test_tree_gpu import _attend, _batch, _dt

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


def _code(x):
    return int(np.flatnonzero(ref.code_values()[:127] == abs(x))[0]) | (128 if x < 0 else 0)


def _cache_of(sd, dtype, n, ps, large, w, below, code):
    """n keys: those in `large` score 0 and have values of 2^w; the others score `below` log2 units less (of a row of q that starts
    with 1) and have the least scale, and codes `code`."""
    import torch
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    pages = n // ps
    k, v, ks, vs = u8(pages, ps, 1, 128), u8(pages, ps, 1, 128), u8(pages, 1, ps) + 127, u8(pages, 1, ps)
    large = large.view(pages, ps)
    k[..., 0, 0] = torch.where(large, 0, _code(-below)).to(torch.uint8)
    v[:, :, 0] = torch.where(large, 0x38, code).to(torch.uint8)[..., None]
    vs[:, 0] = torch.where(large, 127 + w, 127 + ref.least(dtype)).to(torch.uint8)
    return sd.PagedCache8(k, ks, v, vs, dtype=_dt(dtype)), _batch(sd, [list(range(pages))], [0, 1], [n], ps)


FAR = [
    # w, log2 units below, keys.  The shares of the small ones: from 2^-8 to 2^4 of the large one's together
    (7, 7, 4_096), (7, 8, 512), (7, 18, 131_072), (7, 5, 128), (0, 14, 65_536), (0, 18, 262_144), (0, 20, 16_384), (-8, 26, 262_144),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["first", "last", "middle"])
@pytest.mark.parametrize("case", FAR)
def test_small_values_count_in_the_sum(sd, case, order, dtype):
    """One key of a large value among keys of zeros (in its tile, and in those before and behind it, in the other stream's and in
    other CTAs' parts)."""
    import torch
    w, below, n = case
    if dtype == "f16":
        w = min(w, 7)
    large = torch.zeros(n, dtype=torch.bool, device="cuda")
    large[{"first": 0, "last": n - 1, "middle": n // 2 + 5}[order]] = True
    cache, b = _cache_of(sd, dtype, n, 64, large, w, below, 0)
    q = torch.zeros((1, 3, 128), dtype=_dt(dtype), device="cuda")
    q[0, :, 0] = torch.tensor([1.0, 0.5, 2.0])            # scores below, below / 2, 2 * below
    out, lse = _attend(sd, q, cache, b, None, math.log(2.0), 0, 1, True)
    scale = float(np.float32(math.log(2.0)))
    for row, x in enumerate((1.0, 0.5, 2.0)):
        z = 1.0 + (n - 1) * math.exp(-scale * below * x)
        # out: a 16-bit rounding of it and one of the weight; exponents of up to 2^8 rounded twice in fp32, 2^-16 each,
        # and sums of up to 2^8 terms a thread: less than 2^-13 in all
        tol = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -11) + 2.0 ** -11 + 2.0 ** -13
        got = out[0, row].double()
        assert ((got - 2.0 ** w / z).abs() <= tol * 2.0 ** w / z + (2.0 ** -25 if dtype == "f16" else 0)).all(), (got[0].item(), 2.0 ** w / z)
        assert abs(float(lse[0, row]) - math.log(z)) <= 2.0 ** -14 + 2.0 ** -20 * math.log(z)


@pytest.mark.parametrize("order", ["first", "last", "tiles in turn", "at random"])
@pytest.mark.parametrize("w,below", [(7, 6), (7, 15), (0, 15), (-60, 15), (-90, 3)])
def test_values_of_both_kinds(sd, w, below, order):
    """Many keys of either kind, the small ones not zero; one token and many parts of an item."""
    import torch
    for n in (256, 32_768):
        i = torch.arange(n, device="cuda")
        large = {"first": i < n // 4, "last": i >= n - n // 4, "tiles in turn": i // 128 % 2 == 0,
                 "at random": torch.rand(n, device="cuda", generator=torch.Generator("cuda").manual_seed(n)) < 0.01}[order].clone()
        large[n // 3] = True
        cache, b = _cache_of(sd, "bf16", n, 16, large, w, below, 0x7E)      # 448
        q = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
        q[0, :, 0] = torch.tensor([1.0, -1.0])            # the second row: the small ones lie above
        out, lse = _attend(sd, q, cache, b, None, math.log(2.0), 0, 1, True)
        scale, m = float(np.float32(math.log(2.0))), int(large.sum())
        for row, x in enumerate((1.0, -1.0)):
            e = math.exp(-scale * below * x)
            z = m + (n - m) * e
            want = (m * 2.0 ** w + (n - m) * e * 448 * 2.0 ** -120) / z
            got = out[0, row].double()
            assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13) * want).all(), (n, row, got[0].item(), want)
            assert abs(float(lse[0, row]) - math.log(z)) <= 2.0 ** -14 + 2.0 ** -20 * math.log(z)


@pytest.mark.parametrize("n", [1, 192, 100_032, 250_048])
def test_values_all_of_the_least_scale(sd, n):
    """The output is as small as the values, and as exact as any."""
    import torch
    n_pages = -(-n // 64) * 64
    large = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
    cache, _ = _cache_of(sd, "bf16", n_pages, 64, large, 0, 3, 0x7E)
    b = _batch(sd, [list(range(n_pages // 64))], [0, 1], [n], 64)
    q = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    q[0, 1, 0] = 1.0
    out, lse = _attend(sd, q, cache, b, None, math.log(2.0), 0, 1, True)
    # all weights alike: a 16-bit rounding of the output, one of a weight, and sums as above
    assert ((out.double() - 448 * 2.0 ** -120).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13) * 448 * 2.0 ** -120).all(), out[0, :, 0]
    for row, t in enumerate((0.0, -3 * float(np.float32(math.log(2.0))))):
        assert abs(float(lse[0, row]) - t - math.log(n)) <= 2.0 ** -14 + 2.0 ** -20 * math.log(max(n, 2))
