"""Rounds of trees and the 8-bit cache on the GPU, against plain float64 forms
(tests/tree_ref.py).  Needs a GPU."""
from __future__ import annotations

import numpy as np
import pytest

from tests import tree_ref as ref

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


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _dt(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float16


def _cu(sizes):
    return [0] + np.cumsum(sizes).tolist()


def _batch(sd, table, cu, seq, ps):
    return sd.PagedBatch(_i32(table).view(len(seq), -1), _i32(cu), _i32(seq), page_size=ps)


# ---- plan ---------------------------------------------------------------------

@pytest.mark.parametrize("sizes,words,pad,chain", [
    ([1], 1, 0, False), ([16], 1, 3, False), ([64, 0, 33, 2], 2, 0, False), ([256], 8, 1, True), ([256, 255], 8, 0, False),
    ([40, 3], 1, 0, False), ([300, 5], 8, 7, False), ([7] * 400, 1, 2, False), ([0, 0], 1, 4, False)])
def test_plan(sd, sizes, words, pad, chain):
    import torch
    rng = np.random.default_rng(sum(sizes) + words)
    cu = _cu(sizes)
    tokens = cu[-1] + pad
    parents = [p for n in sizes for p in ref.random_parents(rng, n, chain=chain)[:n]] + [5] * pad
    for t in rng.integers(0, tokens, 3).tolist() if len(sizes) > 1 else []:
        parents[t] = int(rng.choice([-7, 1 << 30, 255, -(1 << 31)]))     # nodes without a parent
    seq = [n + int(rng.integers(0, 100_000)) for n in sizes]
    b = _batch(sd, [[0]] * len(sizes), cu, seq, 16)
    masks = torch.full((tokens, words), -5, dtype=torch.int32, device="cuda")
    positions = torch.full((tokens,), -5, dtype=torch.int32, device="cuda")
    sd.spec_tree_plan(_i32(parents), b, masks, positions)
    m, p = ref.plan(parents, cu, seq, tokens, words)
    assert np.array_equal(masks.cpu().numpy().view(np.uint32), m)
    assert positions.cpu().tolist() == p.tolist()


# ---- attention ------------------------------------------------------------------

def _cache(sd, k, v, dtype, eight, garbage=True, seed=0):
    """Keys and values float64 [pages, ps, heads, dim], NaN where nothing is written, in a cache;
    (cache, the values that it holds)."""
    import torch
    rng = np.random.default_rng(seed)
    if not eight:
        t = [torch.tensor(x, device="cuda").to(_dt(dtype)) for x in (k, v)]
        return sd.PagedCache(*t), [x.double().cpu().numpy() for x in t]
    parts, held = [], []
    for x in (k, v):
        there = ~np.isnan(x[..., 0])
        codes = rng.integers(0, 256, x.shape).astype(np.uint8)           # what is unwritten holds anything
        scales = rng.integers(0, 256, x.shape[:-1]).astype(np.uint8)
        codes[there], scales[there] = ref.quantise(x[there], dtype)
        parts += [torch.tensor(codes, device="cuda"), torch.tensor(scales.transpose(0, 2, 1).copy(), device="cuda")]
        held.append(np.where(there[..., None], ref.values(codes, scales), np.nan))
    return sd.PagedCache8(*parts, dtype=_dt(dtype)), held


def _step(sizes, ctx, hk, group, dim, ps, dtype, seed, spare=3, window=0):
    rng = np.random.default_rng(seed)
    seq = [c + n for c, n in zip(ctx, sizes)]
    need = [-(-max(s, 0) // ps) for s in seq]
    pages, most = sum(need) + spare, max(max(need), 1)
    perm = rng.permutation(pages)
    table = np.full((len(sizes), most), -1, dtype=np.int64)
    at = 0
    for lane, n in enumerate(need):
        table[lane, :n] = perm[at:at + n]
        at += n
    k, v = (np.full((pages, ps, hk, dim), np.nan) for _ in range(2))
    for lane, s in enumerate(seq):
        lo = max(0, ctx[lane] - window + 1) if window else 0
        j = np.arange(lo, max(s, lo))
        for x in (k, v):
            # vectors of different sizes, so that scales differ
            x[table[lane][j // ps], j % ps] = rng.standard_normal((len(j), hk, dim)) * 2.0 ** rng.integers(-3, 3, (len(j), hk, 1))
    import torch
    q = torch.tensor(rng.standard_normal((sum(sizes), hk * group, dim)), device="cuda").to(_dt(dtype))
    return seq, table, k, v, q


def _attend(sd, q, cache, batch, masks, scale, window, max_new, eight):
    import torch
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    ws = sd.new_attention_workspace()
    if masks is None:
        f = sd.spec_paged_attention8 if eight else sd.spec_paged_attention
        f(q, cache, batch, scale, out, lse, ws, window=window, max_new=max_new)
    else:
        f = sd.spec_tree_attention8 if eight else sd.spec_tree_attention
        f(q, cache, batch, masks, scale, out, lse, ws, window=window, max_new=max_new)
    torch.cuda.synchronize()
    assert sd.spec_device_status() is None
    return out, lse


def _check(got, lse, want):
    out, lw, ob, lb = want
    g, gl = got.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = ~np.isnan(lw)
    assert np.isfinite(g[rows]).all()
    off = np.abs(g - out)[rows] - ob[rows]              # (a row without keys: 0 of 0)
    assert (off <= 0).all(), off.max()
    empty = np.isneginf(lw)
    assert np.array_equal(np.isneginf(gl) & rows, empty) and (g[empty] == 0).all()
    fine = rows & ~empty
    assert (np.abs(gl[fine] - lw[fine]) <= lb[fine]).all()


TREES = [
    # sizes, cached, kv heads, group, dim, page, dtype, window
    ([1], [0], 1, 1, 64, 16, "bf16", 0),
    ([16], [100], 2, 4, 128, 16, "bf16", 0),
    ([16], [1_013], 2, 4, 128, 16, "f16", 0),
    ([64, 0, 17, 2], [500, 20, 0, 130], 2, 3, 128, 32, "bf16", 0),
    ([64], [127], 1, 8, 128, 64, "bf16", 0),                 # nodes across a tile's end, two row tiles
    ([33, 5], [95, 3_001], 1, 8, 64, 16, "f16", 0),
    ([48, 30], [2_900, 260], 1, 4, 64, 32, "bf16", 300),     # a window
    ([20, 9], [700, 64], 2, 2, 256, 16, "bf16", 0),
    ([70], [190], 1, 4, 256, 128, "f16", 256),
    ([256, 100], [60, 10], 1, 2, 64, 16, "bf16", 0),         # masks of eight words, over two tiles of keys
    ([5] * 40, list(range(0, 400, 10)), 1, 2, 128, 16, "bf16", 0),
]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("case", TREES)
def test_tree_attention(sd, case, eight):
    import torch
    sizes, ctx, hk, group, dim, ps, dtype, window = case
    rng = np.random.default_rng(sum(sizes) + dim)
    seq, table, k, v, q = _step(sizes, ctx, hk, group, dim, ps, dtype, seed=dim + len(sizes), window=window)
    cache, (kk, vv) = _cache(sd, k, v, dtype, eight)
    cu = _cu(sizes)
    words = -(-max(sizes) // 32)
    parents = [p for n in sizes for p in ref.random_parents(rng, n, deep=10)[:n]]
    b = _batch(sd, table.tolist(), cu, seq, ps)
    masks = torch.empty((cu[-1], words), dtype=torch.int32, device="cuda")
    positions = torch.empty(cu[-1], dtype=torch.int32, device="cuda")
    sd.spec_tree_plan(_i32(parents), b, masks, positions)
    scale = dim ** -0.5
    want = ref.attention(q.double().cpu().numpy(), kk, vv, table, cu, seq, masks.cpu().numpy().view(np.uint32), scale, window, dtype)
    for max_new in (0, max(sizes)):
        got, lse = _attend(sd, q, cache, b, masks, scale, window, max_new, eight)
        _check(got, lse, want)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("ctx", [0, 1, 40, 128])
def test_masks_of_any_bits(sd, ctx, eight):
    """Bits that are no tree's: rows that see nothing, bits above the row's own node, which do not count."""
    import torch
    n, dim, ps, dtype = 50, 64, 16, "bf16"
    rng = np.random.default_rng(ctx)
    seq, table, k, v, q = _step([n], [ctx], 1, 3, dim, ps, dtype, seed=ctx)
    cache, (kk, vv) = _cache(sd, k, v, dtype, eight)
    masks = rng.integers(0, 1 << 32, (n, 2), dtype=np.uint64).astype(np.uint32)
    masks[3] = masks[7] = masks[49] = 0
    masks[20] = 0xFFFFFFFF
    masks[5] = [~np.uint32((2 << 5) - 1), 0xFFFFFFFF]        # only bits above node 5
    cu = [0, n]
    want = ref.attention(q.double().cpu().numpy(), kk, vv, table, cu, seq, masks, 0.125, 0, dtype)
    b = _batch(sd, table.tolist(), cu, seq, ps)
    got, lse = _attend(sd, q, cache, b, torch.tensor(masks.view(np.int32), device="cuda"), 0.125, 0, n, eight)
    _check(got, lse, want)


def test_chain_is_causal(sd):
    """A chain's masks give what the causal call gives, bit by bit where both take the same tiles."""
    import torch
    sizes, ctx, hk, group, dim, ps, dtype = [30, 9], [500, 77], 2, 4, 128, 16, "bf16"
    seq, table, k, v, q = _step(sizes, ctx, hk, group, dim, ps, dtype, seed=3)
    cu = _cu(sizes)
    b = _batch(sd, table.tolist(), cu, seq, ps)
    masks = torch.empty((cu[-1], 1), dtype=torch.int32, device="cuda")
    positions = torch.empty(cu[-1], dtype=torch.int32, device="cuda")
    sd.spec_tree_plan(_i32([i - 1 for n in sizes for i in range(n)]), b, masks, positions)
    for eight in (False, True):
        cache, _ = _cache(sd, k, v, dtype, eight)
        a, la = _attend(sd, q, cache, b, masks, 0.09, 0, 30, eight)
        c, lc = _attend(sd, q, cache, b, None, 0.09, 0, 30, eight)
        assert torch.equal(a, c) and torch.equal(la, lc)


CHUNKS = [
    ([1], [0], 1, 1, 64, 16, "bf16", 0), ([1], [1_013], 2, 4, 128, 16, "bf16", 0), ([1] * 9, list(range(0, 900, 100)), 2, 8, 128, 64, "bf16", 0),
    ([8, 3, 0, 16], [500, 0, 9, 2_000], 2, 4, 128, 32, "f16", 0), ([200], [300], 1, 4, 128, 128, "bf16", 0),
    ([130, 1], [77, 4_000], 1, 2, 64, 16, "bf16", 100), ([100, 20], [50, 700], 1, 2, 256, 64, "f16", 0),
    ([7], [9_000], 1, 8, 256, 16, "bf16", 2_048), ([16], [20_000], 1, 8, 128, 128, "bf16", 0), ([300], [0], 2, 1, 64, 32, "f16", 0),
]


@pytest.mark.parametrize("case", CHUNKS)
def test_attention8(sd, case):
    sizes, ctx, hk, group, dim, ps, dtype, window = case
    seq, table, k, v, q = _step(sizes, ctx, hk, group, dim, ps, dtype, seed=dim + ps, window=window)
    cache, (kk, vv) = _cache(sd, k, v, dtype, True)
    cu = _cu(sizes)
    want = ref.attention(q.double().cpu().numpy(), kk, vv, table, cu, seq, None, dim ** -0.5, window, dtype)
    b = _batch(sd, table.tolist(), cu, seq, ps)
    for max_new in (0, max(sizes)):
        got, lse = _attend(sd, q, cache, b, None, dim ** -0.5, window, max_new, True)
        _check(got, lse, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_code_and_scale_widens(sd, dtype):
    """One key a lane: the output is its value vector, which holds every code at each scale."""
    import torch
    scales = list(range(113, 135)) + ([7, 8, 50, 100] if dtype == "bf16" else [])
    codes = [c for c in range(256) if c & 127 != 127] + [0, 0]
    lanes, dim, ps = len(scales), 256, 16
    v = np.zeros((lanes, ps, 1, dim), np.uint8)
    v[:, 0, 0] = codes
    vs = np.full((lanes, 1, ps), 127, np.uint8)
    vs[:, 0, 0] = scales
    z, zs = np.zeros_like(v), np.full_like(vs, 127)
    t = lambda x: torch.tensor(x, device="cuda")  # noqa: E731
    cache = sd.PagedCache8(t(z), t(zs), t(v), t(vs), dtype=_dt(dtype))
    b = _batch(sd, [[i] for i in range(lanes)], list(range(lanes + 1)), [1] * lanes, ps)
    q = torch.zeros((lanes, 1, dim), dtype=_dt(dtype), device="cuda")
    out, _ = _attend(sd, q, cache, b, None, 1.0, 0, 1, True)
    want = torch.tensor(ref.code_values()[codes] * 2.0 ** (np.array(scales, np.float64)[:, None] - 127)).to(_dt(dtype))
    got = out[:, 0].cpu()
    # (the product of a weight of 1 and a subnormal 16-bit value may be flushed by the tensor cores: compare what is normal)
    normal = want.double().abs() >= torch.finfo(_dt(dtype)).tiny
    assert torch.equal(got[normal], want[normal]) or (got.double()[normal] - want.double()[normal]).abs().max() == 0
    assert (got.double()[~normal] - want.double()[~normal]).abs().max() < torch.finfo(_dt(dtype)).tiny


def test_no_number_reads_as_nan(sd):
    """A key that is no number makes the rows that see it NaN, and no other."""
    import torch
    n, ctx, dim, ps = 4, 30, 64, 16
    seq, table, k, v, q = _step([n], [ctx], 1, 2, dim, ps, "bf16", seed=4)
    cache, _ = _cache(sd, k, v, "bf16", True)
    new = torch.randn((1, 1, dim), device="cuda").to(torch.bfloat16)
    bad = new.clone()
    bad[0, 0, 5] = float("inf")
    at = ctx + 2
    sd.spec_paged_store8(bad, new, torch.tensor([int(table[0][at // ps]) * ps + at % ps], device="cuda"), cache)
    b = _batch(sd, table.tolist(), [0, n], seq, ps)
    out, _ = _attend(sd, q, cache, b, None, 0.125, 0, n, True)
    nan = torch.isnan(out).flatten(1)
    assert not nan[:2].any() and nan[2:].all()


# ---- store ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,dim,ps,tokens,order", [(1, 16, 1, 1, "nhd"), (2, 64, 16, 33, "nhd"), (3, 128, 7, 70, "hnd"),
                                                       (2, 256, 64, 9, "nhd"), (5, 48, 16, 19, "hnd"), (1, 240, 16, 5, "nhd")])
def test_store(sd, dtype, heads, dim, ps, tokens, order):
    import torch
    rng = np.random.default_rng(heads * 100 + dim)
    pages = -(-tokens * 2 // ps) + 2
    shape = (pages, ps, heads, dim) if order == "nhd" else (pages, heads, ps, dim)
    codes = [torch.tensor(rng.integers(0, 256, shape).astype(np.uint8), device="cuda") for _ in range(2)]
    view = [x if order == "nhd" else x.transpose(1, 2) for x in codes]
    scales = [torch.tensor(rng.integers(0, 256, (pages, heads, ps)).astype(np.uint8), device="cuda") for _ in range(2)]
    cache = sd.PagedCache8(view[0], scales[0], view[1].view(torch.float8_e4m3fn), scales[1], dtype=_dt(dtype))
    x = rng.standard_normal((tokens, heads * 3, dim)) * 2.0 ** rng.integers(-20 if dtype == "bf16" else -9, 10, (tokens, heads * 3, 1))
    x[0, heads] = 0
    x[0, heads, 3] = -0.0
    if tokens > 4:
        top = float(torch.finfo(_dt(dtype)).max)
        x[1, heads, 0], x[2, heads, 1], x[3, heads, 2], x[3, 2 * heads, 2] = np.inf, np.nan, top, 57_344
        x[4, heads] = np.ldexp(rng.standard_normal(dim), -130 if dtype == "bf16" else -18)     # subnormals
    qkv = torch.tensor(x, device="cuda").to(_dt(dtype))
    nk, nv = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    slots = torch.tensor(rng.permutation(pages * ps)[:tokens], device="cuda")
    if tokens > 6:
        slots[5], slots[6] = -1, pages * ps
    want = [v.cpu().numpy().copy() for v in view], [s.cpu().numpy().copy() for s in scales]
    for i, new in enumerate((nk, nv)):
        c, e = ref.quantise(new.double().cpu().numpy(), dtype)
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < pages * ps:
                want[0][i][s // ps, s % ps] = c[t]
                want[1][i][s // ps, :, s % ps] = e[t]
    sd.spec_paged_store8(nk, nv, slots, cache)
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(scales[i].cpu().numpy(), want[1][i])
        assert np.array_equal(view[i].cpu().numpy(), want[0][i])


# ---- verification ---------------------------------------------------------------

def _verify_case(rng, sizes, V, depth, offset=0, kind="normal"):
    import torch
    cu = _cu(sizes)
    tokens = cu[-1]
    x = 3 * rng.standard_normal((tokens, V))
    if kind == "levels":
        x = np.round(x)
    if kind == "flat":
        x[:] = 1.5
    drafts = rng.integers(0, V, tokens)
    parents = [p for n in sizes for p in ref.random_parents(rng, n)[:n]]
    for lane, n in enumerate(sizes):                          # the target agrees with most parents' first child
        for i in range(1, n):
            if kind == "normal" and rng.random() < 0.5:
                x[cu[lane] + parents[cu[lane] + i], drafts[cu[lane] + i]] = 14 + rng.standard_normal()
    buf = torch.zeros(tokens * V + 16, dtype=torch.bfloat16, device="cuda")
    logits = buf[offset:offset + tokens * V].view(tokens, V)
    logits.copy_(torch.tensor(x).to(torch.bfloat16))
    return cu, logits, drafts, parents


VERIFY = [
    # sizes, V, depth, offset, kind
    ([1], 1, 1, 0, "normal"), ([4], 7, 3, 1, "normal"), ([16], 5_000, 15, 3, "normal"), ([3, 0, 20], 1_001, 6, 5, "normal"),
    ([16], 70_001, 5, 7, "levels"), ([2, 2], 33_000, 2, 2, "flat"), ([40] * 20, 9_999, 8, 1, "normal"),
    ([30] * 12, 40_000, 3, 0, "levels"), ([64] * 70, 1_500, 8, 4, "normal"), ([5] * 300, 50, 4, 0, "levels"),
    ([256, 100], 3_001, 20, 0, "normal"), ([8] * 40, 33_333, 7, 6, "flat"), ([300], 2_000, 255, 0, "normal"),
    ([6] * 60, 262_200, 5, 1, "normal"),                     # more than eight CTAs hold at once: pieces
]


@pytest.mark.parametrize("case", VERIFY)
@pytest.mark.parametrize("top_k", [0, 1, 20, 64])
def test_verify(sd, case, top_k):
    import torch
    sizes, V, depth, offset, kind = case
    rng = np.random.default_rng(V + depth)
    cu, logits, drafts, parents = _verify_case(rng, sizes, V, depth, offset, kind)
    sampled, k = top_k > 0, min(max(top_k, 1), V)
    u = rng.random((cu[-1], 2))
    lanes = len(sizes)
    x = logits.double().cpu().numpy()
    args = (x, drafts.tolist(), parents, cu, depth)
    top_p, T = (0.9, 0.8) if kind != "flat" else (0.955, 1.0)
    acc, ids, path, margin = ref.verify(*args, u.tolist(), T, top_p, k) if sampled else ref.verify(*args)
    assert margin > 1e-12                                     # decisions that 64 bits can take
    outs = [torch.full((lanes,), -9, dtype=torch.int32, device="cuda")] + [
        torch.full((lanes, depth + 1), -9, dtype=torch.int32, device="cuda") for _ in range(2)]
    for _ in range(2):                                        # (the tickets are ready for the next call)
        if sampled:
            sd.spec_tree_verify_sampled(logits, _i32(drafts.tolist()), _i32(parents), _i32(cu), lanes, depth, V, T, top_p, k,
                                        torch.tensor(u, device="cuda"), *outs)
        else:
            sd.spec_tree_verify(logits, _i32(drafts.tolist()), _i32(parents), _i32(cu), lanes, depth, V, *outs)
    assert outs[0].cpu().tolist() == acc
    assert outs[1].cpu().tolist() == ids
    assert outs[2].cpu().tolist() == path


@pytest.mark.parametrize("lanes", [1, 60])
def test_chain_is_the_verify_of_a_row(sd, lanes):
    import torch
    rng = np.random.default_rng(lanes)
    gamma, V = 7, 20_000
    cu, logits, drafts, _ = _verify_case(rng, [gamma + 1] * lanes, V, gamma)
    parents = [i - 1 for _ in range(lanes) for i in range(gamma + 1)]
    rows = drafts.reshape(lanes, gamma + 1)
    for lane in range(lanes):
        for i in range(gamma):
            if rng.random() < 0.8:
                logits[lane * (gamma + 1) + i, int(rows[lane, i + 1])] = 15
    flat = _i32(rows[:, 1:].tolist()).contiguous()
    a, c = sd.verify(logits, flat)
    ta, tc, path = sd.tree_verify(logits, _i32(drafts.tolist()), _i32(parents), _i32(cu), gamma)
    assert torch.equal(a, ta) and torch.equal(c, tc)
    for lane, n in enumerate(a.tolist()):
        assert path[lane].tolist() == list(range(n + 1)) + [-1] * (gamma - n)
    u = torch.rand((lanes, gamma + 1, 2), dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    e = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    acc, com = e(lanes), e(lanes, gamma + 1)
    sd.spec_verify_sampled(logits, flat, lanes, gamma, V, 1.0, 0.95, 20, u, acc, com)
    shifted = u.clone()
    shifted[:, 1:, 0] = u[:, :-1, 0]
    ta, tc, _ = sd.tree_verify(logits, _i32(drafts.tolist()), _i32(parents), _i32(cu), gamma, uniforms=shifted.view(-1, 2),
                               top_p=0.95, top_k=20)
    assert torch.equal(acc, ta) and torch.equal(com, tc)


def test_sampled_tokens_follow_the_target(sd):
    """Over a grid of uniforms the first committed token has the target's distribution, whatever the drafts."""
    import torch
    q = np.array([0.5, 0.25, 0.125, 0.125])
    side = 48
    grid = (np.arange(side) + 0.5) / side
    u1, u2, u3 = (x.ravel() for x in np.meshgrid(grid, grid, grid, indexing="ij"))
    lanes = len(u1)
    lanes_at_once = 48 * 48
    counts = np.zeros(4)
    for at in range(0, lanes, lanes_at_once):
        n = lanes_at_once
        cu = list(range(0, 3 * n + 1, 3))
        logits = torch.tensor(np.log(q)).to(torch.bfloat16).repeat(3 * n, 1).cuda()
        drafts, parents = _i32([0, 1, 2] * n), _i32([-1, 0, 0] * n)       # the second and third likeliest tokens
        u = np.zeros((n, 3, 2))
        u[:, 0, 1], u[:, 1, 0], u[:, 2, 0] = u1[at:at + n], u2[at:at + n], u3[at:at + n]
        _, ids, _ = sd.tree_verify(logits, drafts, parents, _i32(cu), 1, uniforms=torch.tensor(u.reshape(-1, 2), device="cuda"), top_k=4)
        counts += np.bincount(ids[:, 0].cpu().numpy(), minlength=4)
    e = np.exp(torch.tensor(np.log(q)).to(torch.bfloat16).double().numpy())
    # each of the (at most three) comparisons of a token moves by at most one step of its grid
    assert np.abs(counts / lanes - e / e.sum()).max() <= 3 / side


# ---- commit ----------------------------------------------------------------------

@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("sizes,ctx,hk,dim,ps,depth,order", [
    ([5], [0], 1, 64, 16, 3, "nhd"), ([64, 0, 30, 1], [100, 7, 15, 3], 3, 128, 16, 8, "nhd"),
    ([256], [40], 2, 64, 8, 255, "hnd"), ([20] * 50, list(range(50)), 2, 256, 32, 6, "nhd"), ([33, 33], [1, 2], 5, 48, 7, 12, "hnd")])
def test_commit(sd, eight, sizes, ctx, hk, dim, ps, depth, order):
    import torch
    rng = np.random.default_rng(depth + dim)
    seq = [c + n for c, n in zip(ctx, sizes)]
    need = [-(-s // ps) for s in seq]
    pages = sum(need) + 2
    perm = rng.permutation(pages)
    table = np.full((len(sizes), max(need)), -1)
    at = 0
    for lane, n in enumerate(need):
        table[lane, :n] = perm[at:at + n]
        at += n
    shape = (pages, ps, hk, dim) if order == "nhd" else (pages, hk, ps, dim)
    if eight:
        made = [torch.tensor(rng.integers(0, 256, shape).astype(np.uint8), device="cuda") for _ in range(2)]
        scales = [torch.tensor(rng.integers(0, 256, (pages, hk, ps)).astype(np.uint8), device="cuda") for _ in range(2)]
    else:
        made = [torch.tensor(rng.integers(-9999, 9999, shape).astype(np.int16), device="cuda").view(torch.bfloat16) for _ in range(2)]
        scales = []
    views = [x if order == "nhd" else x.transpose(1, 2) for x in made]
    cache = sd.PagedCache8(views[0], scales[0], views[1], scales[1]) if eight else sd.PagedCache(*views)
    # paths: increasing; one ends early at an entry that is none, one says more than depth
    path = np.full((len(sizes), depth + 1), -1)
    accept = []
    for lane, n in enumerate(sizes):
        a = int(rng.integers(0, min(depth, max(n - 1, 0)) + 1))
        path[lane, :a + 1] = [0] + sorted(rng.choice(np.arange(1, n), a, replace=False).tolist()) if n else -1
        accept.append(a)
    accept[0] = min(depth, sizes[0] - 1)
    path[0, :accept[0] + 1] = [0] + sorted(rng.choice(np.arange(1, sizes[0]), accept[0], replace=False).tolist())
    if len(sizes) > 10:
        path[3, 2:] = [0] * (depth - 1)
        accept[3] = depth + 5
    raw = [x.view(torch.int16) if not eight else x for x in views]
    want = [x.cpu().numpy().copy() for x in raw + scales]
    after = []
    for lane, n in enumerate(sizes):
        moves = 0
        if n:
            for i in range(1, min(accept[lane], depth) + 1):
                node = int(path[lane, i])
                if not i <= node < n:
                    break
                (fp, fr), (tp, tr) = (divmod(ctx[lane] + x, ps) for x in (node, i))
                for j in range(2):
                    want[j][table[lane][tp], tr] = want[j][table[lane][fp], fr]
                for x in want[2:]:
                    x[table[lane][tp], :, tr] = x[table[lane][fp], :, fr]
                moves = i
        after.append(ctx[lane] + 1 + moves if n else ctx[lane])
    context = torch.full((len(sizes),), -9, dtype=torch.int32, device="cuda")
    f = sd.spec_tree_commit8 if eight else sd.spec_tree_commit
    f(cache, _batch(sd, table.tolist(), _cu(sizes), seq, ps), _i32(path.tolist()), _i32(accept), depth, context)
    assert context.cpu().tolist() == after
    for got, w in zip(raw + scales, want):
        assert np.array_equal(got.cpu().numpy(), w)


def test_commit_skips_pages_that_are_none(sd):
    import torch
    k = torch.arange(4 * 4 * 8, dtype=torch.int16, device="cuda").view(4, 4, 1, 8).view(torch.bfloat16)
    cache = sd.PagedCache(k.clone(), k.clone())
    b = _batch(sd, [[0, -1, 9, 2]], [0, 16], [16], 4)
    # into page 0 from pages that are no pages and from page 2 (position 12 on)
    sd.spec_tree_commit(cache, b, _i32([[0, 5, 9, 13]]), _i32([3]), 3)
    want = k.clone()
    want[0, 3] = want[2, 1]
    assert torch.equal(cache.k.view(torch.int16), want.view(torch.int16))


# ---- together ----------------------------------------------------------------------

@pytest.mark.parametrize("eight", [False, True])
def test_a_round_in_a_graph(sd, eight):
    """Plan, masks, store, attention, verify and commit captured on a stream of their own and replayed twice,
    against the same calls one by one."""
    import torch
    g = torch.Generator("cuda").manual_seed(5)
    lanes, nodes, hk, group, dim, ps, V, depth = 6, 20, 2, 4, 64, 16, 8_000, 5
    rng = np.random.default_rng(8)
    parents = _i32([p for _ in range(lanes) for p in ref.random_parents(rng, nodes, deep=depth)])
    drafts = torch.randint(0, V, (lanes * nodes,), generator=g, device="cuda", dtype=torch.int32)
    tokens = lanes * nodes
    k, v = (torch.randn((tokens, hk, dim), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((tokens, hk * group, dim), generator=g, device="cuda").to(torch.bfloat16)
    logits = (3 * torch.randn((tokens, V), generator=g, device="cuda")).to(torch.bfloat16)
    uniforms = torch.rand((tokens, 2), generator=g, device="cuda", dtype=torch.float64)
    for t in range(tokens):
        if t % nodes:
            logits[t - t % nodes + int(parents[t]), int(drafts[t])] = 14.0

    def make():
        shape = (40, ps, hk, dim)
        if eight:
            cache = sd.PagedCache8.create(*shape)
        else:
            cache = sd.PagedCache(*(torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
        b = sd.PagedBatch.create(lanes, 6, tokens, ps)
        b.new_lens.fill_(nodes)
        e = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        s = dict(cache=cache, b=b, free=torch.arange(40, dtype=torch.int32, device="cuda"), cursor=_i32([0]), masks=e(tokens, 1),
                 positions=e(tokens), out=torch.empty_like(q), lse=torch.empty(q.shape[:2], device="cuda"),
                 ws=sd.new_attention_workspace(), acc=e(lanes), ids=e(lanes, depth + 1), path=e(lanes, depth + 1), nxt=e(lanes))
        return s

    def round_(s):
        sd.spec_paged_plan(s["b"], s["free"], s["cursor"])
        sd.spec_tree_plan(parents, s["b"], s["masks"], s["positions"])
        (sd.spec_paged_store8 if eight else sd.spec_paged_store)(k, v, s["b"].slots, s["cache"])
        (sd.spec_tree_attention8 if eight else sd.spec_tree_attention)(q, s["cache"], s["b"], s["masks"], 0.125, s["out"], s["lse"], s["ws"],
                                                                       max_new=nodes)
        sd.spec_tree_verify_sampled(logits, drafts, parents, s["b"].cu_new, lanes, depth, V, 1.0, 0.95, 20, uniforms, s["acc"],
                                    s["ids"], s["path"])
        (sd.spec_tree_commit8 if eight else sd.spec_tree_commit)(s["cache"], s["b"], s["path"], s["acc"], depth, s["nxt"])
        s["b"].context_lens.copy_(s["nxt"])
        s["b"].held.copy_(s["b"].held_out)
        s["cursor"].copy_(s["b"].info[1:2])

    a, c = make(), make()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        round_(make())                                       # (warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        round_(c)
    for _ in range(2):
        round_(a)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "lse", "acc", "ids", "path", "nxt", "masks", "positions"):
            assert torch.equal(a[name], c[name]), name
        x, y = a["cache"], c["cache"]
        assert torch.equal(x.k.view(torch.uint8), y.k.view(torch.uint8)) and torch.equal(x.v.view(torch.uint8), y.v.view(torch.uint8))
    # (a lane commits a token a round at least)
    assert int(a["nxt"].min()) >= 2 and int(a["nxt"].max()) > 2 and sd.spec_device_status() is None
