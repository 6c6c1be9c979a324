"""Attention in fp16 where one key outweighs each of very many others: their
weights are far below fp16's smallest number, their sum is not.  Needs a GPU.

Bound: the weights enter the second product in fp16, scaled so that the
largest is at least 2^7 (a reference lags the row's maximum by at most 2^8
more, which makes the stored weights larger).  A weight then rounds to 2^-11 of
itself, or, below 2^-14, to 2^-25 absolute, which is 2^-32 of the largest.
Scores carry an fp32 error of E = 2^-20 * scale * max_j sum_i |q_i k_ji|, which moves a
weight and the sum by E relative each, exponentials and sums are good to
2^-18, and the result rounds once more:
    err = (2^-11 + 2 E + 2^-18) * sum_j w_j |v_j| + 2^-32 * max w * sum_j |v_j|,
    |out - o| <= 2^-11 (|o| + err) + err + 2^-25."""
from __future__ import annotations

import numpy as np
import pytest

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


def _run(sd, keys, lanes, dim, drop, at, seed, dtype="f16"):
    """`lanes` lanes that share one context of `keys` keys: the key at `at` has the
    score 0, the others lie about `drop` below it in log2, spread by 0.3.  The
    dominant key's value is small, the others' are about 1."""
    import torch
    dt = torch.float16 if dtype == "f16" else torch.bfloat16
    rng = np.random.default_rng(seed)
    ps = 64
    k, v = np.zeros((keys, dim)), 1.0 + 0.25 * rng.standard_normal((keys, dim))
    q = np.zeros((lanes, dim))
    q[:, 0] = 8.0
    k[:, 0] = -(drop + 0.3 * rng.standard_normal(keys)) * np.log(2.0)
    k[at, 0] = 0.0
    v[at] = 0.01
    to = lambda x: torch.from_numpy(x).to(dt).cuda()  # noqa: E731
    kt, vt, qt = to(k).view(-1, ps, 1, dim), to(v).view(-1, ps, 1, dim), to(q).view(lanes, 1, dim)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(keys // ps, dtype=torch.int32, device="cuda").expand(lanes, -1).contiguous()
    batch = sd.PagedBatch(table, i32(list(range(lanes + 1))), i32([keys] * lanes), page_size=ps)
    out, lse = sd.paged_attention(qt, sd.PagedCache(kt, vt), batch, scale=1.0 / 8.0, max_new=1)
    torch.cuda.synchronize()
    sd.spec_device_status()
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    kk, vv, qq = f(kt).reshape(keys, dim), f(vt).reshape(keys, dim), f(qt).reshape(lanes, dim)
    s = kk @ qq[0] / 8.0
    m = s.max()
    w = np.exp(s - m)
    z = w.sum()
    w /= z
    o, A, E = w @ vv, w @ np.abs(vv), 2.0 ** -20 / 8.0 * (np.abs(kk) @ np.abs(qq[0])).max()
    u = 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    err = (u + 2 * E + 2.0 ** -18) * A + (2.0 ** -32 / z * np.abs(vv).sum(0) if dtype == "f16" else 0.0)
    bound = u * (np.abs(o) + err) + err + 2.0 ** -25
    off = np.abs(f(out).reshape(lanes, dim) - o)
    assert (off <= bound).all(), f"out: worst err/bound {(off / bound).max():.2f}; share of the tail {1 - w[at]:.5f}"
    want = m + np.log(z)
    assert (np.abs(f(lse) - want) <= E + 2.0 ** -20 * max(1.0, abs(want))).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("drop", [14.0, 20.0, 24.7, 25.3, 27.0])
@pytest.mark.parametrize("at", [0, 40])
def test_tail_of_a_long_context(sd, dim, drop, at):
    """As many lanes as fill the GPU, so that one CTA works through a lane's
    whole context and all of its weights are taken against one maximum."""
    _run(sd, 16_384, 304, dim, drop, at, seed=int(drop))


@pytest.mark.parametrize("drop", [25.3, 18.0])
def test_tail_in_bf16(sd, drop):
    _run(sd, 16_384, 304, 128, drop, 0, seed=3, dtype="bf16")


@pytest.mark.parametrize("dim", [64, 256])
def test_tail_in_parts(sd, dim):
    """One lane, whose context is cut over the GPU and joined."""
    _run(sd, 65_536, 1, dim, 22.0, 30, seed=5)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("log2", [16, 22, 24, 25, 26])
def test_weights_stay_finite_at_large_scores(sd, dim, log2):
    """Scores of 2^16 to 2^26 (in log2 units) that differ by up to 20: from
    2^24 on fp32 no longer tells them apart to a unit, and the weights with it, but a
    weighted mean of values in [0.5, 1.5] lies there all the same, up to the
    roundings of the weights against their sum and of the result (2^-11 each)."""
    import torch
    rng = np.random.default_rng(log2 + dim)
    keys, lanes, ps = 4_096, 40, 64
    c = np.log2(np.e)
    k, q = np.zeros((keys, dim)), np.zeros((lanes, dim))
    big = 2.0 ** log2 / c
    q[:, 0], k[:, 0] = 2.0 ** (log2 // 2), big / 2.0 ** (log2 // 2)
    q[:, 1], k[:, 1] = 1.0, rng.uniform(0, 20, keys) / c
    to = lambda x: torch.from_numpy(x).to(torch.float16).cuda()  # noqa: E731
    v = to(rng.uniform(0.5, 1.5, (keys, dim))).view(-1, ps, 1, dim)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(keys // ps, dtype=torch.int32, device="cuda").expand(lanes, -1).contiguous()
    batch = sd.PagedBatch(table, i32(list(range(lanes + 1))), i32([keys] * lanes), page_size=ps)
    assert np.isfinite(k.astype(np.float16)).all() and np.isfinite(q.astype(np.float16)).all()
    out, lse = sd.paged_attention(to(q).view(lanes, 1, dim), sd.PagedCache(to(k).view(-1, ps, 1, dim), v), batch, scale=1.0, max_new=1)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert float(out.min()) >= 0.5 * (1 - 2.0 ** -9) and float(out.max()) <= 1.5 * (1 + 2.0 ** -9)
