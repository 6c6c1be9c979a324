"""The paged cache on the GPU -- plan, store and attention -- against plain
float64 forms (tests/paged_ref.py).  Needs a GPU."""
from __future__ import annotations

import numpy as np
import pytest

from tests import paged_ref as ref

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


# ---- plan -------------------------------------------------------------------

def _run_plan(sd, ctx, new, held, table, free, cursor, ps, tokens):
    import torch
    lanes = len(ctx)
    b = sd.PagedBatch(_i32(table).view(lanes, -1) if lanes else torch.zeros((0, 4), dtype=torch.int32, device="cuda"),
                      torch.full((lanes + 1,), -9, dtype=torch.int32, device="cuda"), _i32([-9] * lanes),
                      page_size=ps, context_lens=_i32(ctx), new_lens=_i32(new), held=_i32(held),
                      held_out=_i32([-9] * lanes), positions=_i32([-9] * tokens),
                      slots=torch.full((tokens,), -9, dtype=torch.int64, device="cuda"), info=_i32([-9] * 4))
    for _ in range(2):    # repeating the call repeats its results
        sd.spec_paged_plan(b, _i32(free), None if cursor is None else _i32([cursor]))
    torch.cuda.synchronize()
    got = [b.block_table, b.cu_new, b.seq_lens, b.held_out, b.positions, b.slots, b.info]
    return [x.cpu().tolist() for x in got]


@pytest.mark.parametrize("lanes,ps,most,new_hi,ctx_hi,free,pad", [
    (1, 16, 4, 1, 0, 4, 0), (1, 1, 9, 3, 5, 20, 2), (3, 16, 10, 20, 100, 60, 7), (8, 64, 8, 8, 400, 40, 0),
    (33, 7, 30, 60, 100, 500, 100), (513, 32, 12, 9, 300, 6_000, 3), (1_500, 16, 6, 40, 50, 9_000, 0),
    (8, 16, 6, 50, 100, 9, 4),            # too few free pages
    (8, 16, 3, 50, 100, 400, 4),          # table rows too short
    (4_096, 128, 3, 3, 250, 9_000, 11), (5, 16, 8, 40, 40, 0, 0)])
def test_plan(sd, lanes, ps, most, new_hi, ctx_hi, free, pad):
    rng = np.random.default_rng(lanes * 131 + ps)
    new = rng.integers(0, new_hi + 1, lanes)
    ctx = rng.integers(0, ctx_hi + 1, lanes)
    if lanes > 4:
        new[1], ctx[2], new[3] = 0, 0, -4
    held = np.minimum(-(-np.maximum(ctx, 0) // ps), most)
    held[lanes // 2] = min(most, held[lanes // 2] + 1)        # a page kept from a rejected tail
    pool = rng.permutation(int(held.sum()) + free + 5)
    table = np.full((lanes, most), -1)
    at = 0
    for l in range(lanes):
        table[l, :held[l]] = pool[at:at + held[l]]
        at += held[l]
    cursor = None if lanes % 2 else 2
    fl = pool[at:at + free + (cursor or 0)].tolist()
    tokens = int(np.maximum(new, 0).sum()) + pad
    args = (ctx.tolist(), new.tolist(), held.tolist(), table.tolist(), fl)
    got = _run_plan(sd, *args, cursor, ps, tokens)
    want = ref.plan(*args, cursor or 0, ps, tokens)
    for name, g, w in zip(("table", "cu_new", "seq_lens", "held", "positions", "slots", "info"), got, want):
        assert g == [list(r) for r in w] if name == "table" else g == list(w), name


def test_plan_of_no_lanes_and_small_buffers(sd):
    got = _run_plan(sd, [], [], [], [], [3], None, 16, 5)
    assert got[1] == [0] and got[4] == [0] * 5 and got[5] == [-1] * 5 and got[6] == [0, 0, 0, 0]
    # fewer token entries than tokens: what fits is written, the total is told
    got = _run_plan(sd, [5], [40], [1], [[7, -1, -1]], [1, 2], None, 16, 10)
    assert got[5] == [7 * 16 + p for p in range(5, 15)] and got[6] == [40, 2, 0, 0] and got[1] == [0, 40]


# ---- store ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,dim,ps,tokens,order", [(1, 8, 1, 1, "nhd"), (2, 64, 16, 33, "nhd"),
                                                       (8, 128, 7, 257, "hnd"), (3, 256, 64, 100, "nhd"),
                                                       (5, 40, 16, 19, "hnd")])
def test_store(sd, dtype, heads, dim, ps, tokens, order):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = torch.Generator(device="cuda").manual_seed(heads * 100 + dim)
    pages = -(-tokens * 2 // ps) + 2
    shape = (pages, ps, heads, dim) if order == "nhd" else (pages, heads, ps, dim)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(2))
    kc, vc = (k, v) if order == "nhd" else (k.transpose(1, 2), v.transpose(1, 2))
    cache = sd.PagedCache(kc, vc)
    qkv = torch.randn((tokens, heads * 3, dim), generator=g, device="cuda").to(dt)
    nk, nv = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:tokens]
    if tokens > 4:
        slots[1], slots[2], slots[4] = -1, pages * ps, 1 << 40     # skipped
    wk, wv = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * ps:
            wk[s // ps, s % ps], wv[s // ps, s % ps] = nk[t], nv[t]
    sd.spec_paged_store(nk, nv, slots, cache)
    torch.cuda.synchronize()
    assert torch.equal(kc.view(torch.int16), wk.view(torch.int16)) and torch.equal(vc.view(torch.int16), wv.view(torch.int16))


# ---- attention --------------------------------------------------------------

def _dt(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float16


def _case(new, ctx, hk, group, dim, ps, dtype, order="nhd", seed=0, spare=3, fill=float("nan"), window=0, sharp=1.0):
    """Inputs of a step.  What no lane may see -- other pages, slots past a
    lane's end, pages before its window -- is `fill`."""
    import torch
    rng = np.random.default_rng(seed)
    lanes, dt = len(new), _dt(dtype)
    seq = [c + n for c, n in zip(ctx, new)]
    need = [-(-s // ps) for s in seq]
    pages, most = sum(need) + spare, max(max(need), 1)
    perm = rng.permutation(pages)
    table = np.full((lanes, most), -1, dtype=np.int64)
    at = 0
    for l, n in enumerate(need):
        table[l, :n] = perm[at:at + n]
        at += n
    shape = (pages, ps, hk, dim) if order == "nhd" else (pages, hk, ps, dim)
    k, v = (torch.full(shape, fill, dtype=dt, device="cuda") for _ in range(2))
    kc, vc = (k, v) if order == "nhd" else (k.transpose(1, 2), v.transpose(1, 2))
    for l in range(lanes):
        lo = max(0, ctx[l] - window + 1) if window else 0
        if new[l] == 0 or seq[l] <= lo:
            continue
        j = np.arange(lo, seq[l])
        pg = torch.from_numpy(table[l][j // ps]).cuda()
        off = torch.from_numpy(j % ps).cuda()
        kc[pg, off] = torch.from_numpy(rng.standard_normal((len(j), hk, dim))).to(dt).cuda()
        vc[pg, off] = torch.from_numpy(rng.standard_normal((len(j), hk, dim))).to(dt).cuda()
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = torch.from_numpy(sharp * rng.standard_normal((cu[-1] + 2, hk * group, dim))).to(dt).cuda()
    return dict(q=q, k=kc, v=vc, table=table, cu=cu, seq=seq, dtype=dtype, window=window)


def _attend(sd, c, q=None, seq=None, max_new=0, ws=None, scale=None):
    import torch
    q = c["q"] if q is None else q
    dim = q.shape[2]
    seq = c["seq"] if seq is None else seq
    cache = sd.PagedCache(c["k"], c["v"])
    batch = sd.PagedBatch(_i32(c["table"].tolist()), _i32(c["cu"]), _i32(seq), page_size=c["k"].shape[1])
    out = torch.full(tuple(q.shape), 7.5, dtype=q.dtype, device="cuda")
    lse = torch.full(tuple(q.shape[:2]), 7.5, dtype=torch.float32, device="cuda")
    ws = sd.new_attention_workspace() if ws is None else ws
    sd.spec_paged_attention(q, cache, batch, dim ** -0.5 if scale is None else scale, out, lse, ws, c["window"], max_new)
    torch.cuda.synchronize()
    sd.spec_device_status()
    return out, lse


def _check(c, out, lse, q=None, seq=None, scale=None):
    q = c["q"] if q is None else q
    seq = c["seq"] if seq is None else seq
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    o, ls, ob, lb = ref.attention(f(q), f(c["k"]), f(c["v"]), c["table"], c["cu"], seq,
                                  q.shape[2] ** -0.5 if scale is None else scale, c["window"], c["dtype"])
    total = c["cu"][-1]
    go, gl = f(out), f(lse)
    assert (go[total:] == 7.5).all() and (gl[total:] == 7.5).all(), "rows past the step's tokens were written"
    go, gl, o, ls, ob, lb = go[:total], gl[:total], o[:total], ls[:total], ob[:total], lb[:total]
    assert np.isfinite(go).all()
    assert (np.abs(go - o) <= ob).all(), f"out: worst err/bound {np.max(np.abs(go - o) / np.maximum(ob, 1e-30)):.3f}"
    none = np.isneginf(ls)
    assert np.array_equal(np.isneginf(gl), none)
    assert (np.abs(gl - ls)[~none] <= lb[~none]).all(), "lse outside its bound"


SHAPES = [
    # new, ctx of each lane
    ([1], [0]), ([1], [1]), ([1], [127]), ([1], [128]), ([1], [300]), ([8], [0]), ([8], [121]), ([5, 0, 1, 16], [0, 40, 129, 77]),
    ([130], [0]), ([257], [3]), ([40, 1, 3], [250, 511, 0]), ([2, 2, 2, 2, 2, 2, 2], [5, 1000, 17, 129, 255, 256, 64]),
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention_shapes(sd, dim, shape):
    new, ctx = SHAPES[shape]
    for i, (hk, group, ps, dtype, order) in enumerate([(2, 4, 16, "bf16", "nhd"), (1, 1, 128, "f16", "hnd"),
                                                       (3, 5, 8, "bf16", "hnd"), (1, 8, 64, "f16", "nhd"),
                                                       (2, 3, 256, "bf16", "nhd")]):
        c = _case(new, ctx, hk, group, dim, ps, dtype, order, seed=shape * 10 + i)
        out, lse = _attend(sd, c, max_new=max(new))
        _check(c, out, lse)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 64, 100, 128, 333])
def test_attention_window(sd, dim, window):
    for new, ctx, ps in (([1, 8, 3], [700, 333, 0], 16), ([150, 2], [130, 1], 64)):
        c = _case(new, ctx, 2, 4, dim, ps, "bf16", seed=window, window=window)
        out, lse = _attend(sd, c, max_new=max(new))
        _check(c, out, lse)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_with_no_key(sd, dim):
    """A seq_len below the chunk leaves its first rows nothing to attend."""
    for new, ctx, seq in (([4, 3], [0, 0], [2, 0]), ([200, 1], [0, 0], [150, 0])):
        c = _case(new, ctx, 1, 4, dim, 16, "bf16")
        out, lse = _attend(sd, c, seq=seq, max_new=max(new))
        _check(c, out, lse, seq=seq)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_hint_does_not_change_what_is_computed(sd, dim):
    c = _case([70, 1], [60, 200], 2, 4, dim, 32, "bf16")
    for max_new in (0, 1, 70, 100_000):
        out, lse = _attend(sd, c, max_new=max_new)
        _check(c, out, lse)


@pytest.mark.parametrize("dim", [64, 128])
def test_large_scores(sd, dim):
    """Sharp softmaxes whose maximum moves a long way from tile to tile."""
    for dtype in ("bf16", "f16"):
        c = _case([9, 33], [900, 700], 1, 4, dim, 16, dtype, seed=5, sharp=12.0)
        # keys that grow along the sequence
        for l, s in enumerate(c["seq"]):
            j = np.arange(s)
            import torch
            pg, off = torch.from_numpy(c["table"][l][j // 16]).cuda(), torch.from_numpy(j % 16).cuda()
            c["k"][pg, off] *= torch.from_numpy(0.2 + j / s).to(c["k"].dtype).cuda()[:, None, None]
        out, lse = _attend(sd, c, max_new=33)
        _check(c, out, lse)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,ctx", [([1], [40]), ([5, 3], [300, 90]), ([2], [9_000]), ([200], [700])])
def test_nan_queries_stay_in_their_rows(sd, dim, new, ctx):
    """A head of a token that is NaN gives NaN for itself and leaves the other rows' bits alone."""
    import torch
    c = _case(new, ctx, 2, 4, dim, 16, "bf16", seed=9)
    out, lse = _attend(sd, c, max_new=max(new))
    _check(c, out, lse)
    q = c["q"].clone()
    gone = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for t in range(0, c["cu"][-1], 3):
        gone[t, t % 8] = gone[t, (t + 5) % 8] = True
    q[gone] = float("nan")
    out2, lse2 = _attend(sd, c, q=q, max_new=max(new))
    assert torch.isnan(out2[gone]).all() and torch.isnan(lse2[gone]).all()
    assert torch.equal(out2[~gone].view(torch.int16), out[~gone].view(torch.int16)) and torch.equal(lse2[~gone], lse[~gone])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_with_no_key_after_nan_parts(sd, dim):
    """An item in parts whose first rows attend nothing, in a workspace where another call's parts were NaN."""
    ws = sd.new_attention_workspace()
    c = _case([300], [40_000], 1, 1, dim, 64, "bf16")
    out, _ = _attend(sd, c, q=c["q"] * float("nan"), max_new=300, ws=ws)
    assert out[:300].isnan().all()
    for seq in (200, 160, 250):
        c = _case([300], [0], 1, 1, dim, 16, "bf16")
        out, lse = _attend(sd, c, seq=[seq], max_new=300, ws=ws)
        _check(c, out, lse, seq=[seq])


def test_strided_queries_and_scale(sd):
    import torch
    c = _case([8, 1], [200, 31], 2, 4, 128, 16, "bf16")
    wide = torch.randn((c["q"].shape[0], 24, 128), device="cuda").to(torch.bfloat16)
    q = wide[:, 4:12]
    out, lse = _attend(sd, c, q=q, scale=0.3)
    _check(c, out, lse, q=q, scale=0.3)
    q = torch.randn((8, c["q"].shape[0], 128), device="cuda").to(torch.bfloat16).transpose(0, 1)   # heads outermost
    out, lse = _attend(sd, c, q=q)
    _check(c, out, lse, q=q)


def test_long_split_context_and_workspace_reuse(sd):
    """Contexts split over many CTAs; the same workspace through calls of different sizes, twice each, equal bits."""
    import torch
    ws = sd.new_attention_workspace()
    for dim, new, ctx in ((128, [1], [20_000]), (64, [16, 3], [9_000, 12_345]), (128, [5, 1, 2], [100, 30_000, 7]),
                          (256, [4], [9_999])):
        c = _case(new, ctx, 1, 2, dim, 64, "bf16")
        out, lse = _attend(sd, c, ws=ws)
        _check(c, out, lse)
        out2, lse2 = _attend(sd, c, ws=ws)
        assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_tiles_per_cta(sd, dim):
    """Runs of many tiles: several items, and several tiles of an item, in every CTA."""
    rng = np.random.default_rng(dim)
    c = _case([3] * 24, rng.integers(0, 2_200, 24).tolist(), 4, 2, dim, 32, "bf16", seed=1)
    out, lse = _attend(sd, c, max_new=3)
    _check(c, out, lse)
    c = _case([2], [70_000], 1, 1, dim, 64, "f16", seed=2)
    out, lse = _attend(sd, c, max_new=2)
    _check(c, out, lse)
    c = _case([700, 1], [900, 1_100], 2, 4, dim, 16, "bf16", seed=3)
    out, lse = _attend(sd, c, max_new=700)
    _check(c, out, lse)
    c = _case([300], [4_000], 2, 3, dim, 128, "f16", seed=4, sharp=6.0)
    out, lse = _attend(sd, c, max_new=300)
    _check(c, out, lse)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_runs_cut_between_items(sd, dim):
    """Enough tiles for every CTA, in items of one to a dozen: runs that begin and end inside items, between them,
    and before an item's first tile."""
    rng = np.random.default_rng(dim + 1)
    step = 64 if dim == 256 else 128
    for lanes, new, most, hk, group in ((40, 2, 9, 2, 4), (24, 1, 12, 3, 1), (9, 200, 5, 2, 4), (150, 3, 4, 1, 2)):
        ctx = (step * most * rng.random(lanes)).astype(int).tolist()
        c = _case([new] * lanes, ctx, hk, group, dim, 32, "bf16", seed=lanes)
        for max_new in (new, 0):
            out, lse = _attend(sd, c, max_new=max_new)
            _check(c, out, lse)


def test_many_lanes(sd):
    rng = np.random.default_rng(3)
    new, ctx = rng.integers(0, 3, 700).tolist(), rng.integers(0, 40, 700).tolist()
    c = _case(new, ctx, 1, 2, 64, 16, "bf16")
    out, lse = _attend(sd, c)
    _check(c, out, lse)


def test_bad_table_entries_read_as_zero(sd):
    import torch
    c = _case([2], [40], 1, 1, 64, 16, "bf16")
    c["table"][0, 1] = 1 << 30
    out, lse = _attend(sd, c)
    c["k"] = torch.cat([c["k"], torch.zeros_like(c["k"][:1])])
    c["v"] = torch.cat([c["v"], torch.zeros_like(c["v"][:1])])
    c["table"][0, 1] = c["k"].shape[0] - 1
    _check(c, out, lse)


def test_offsets_past_32_bits(sd):
    """A cache of more than 2^32 elements, its pages at both ends."""
    import torch
    ps, hk, dim = 16, 8, 128
    pages = (1 << 32) // (ps * hk * dim) + 64
    k = torch.empty((pages, ps, hk, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((pages, ps, hk, dim), dtype=torch.bfloat16, device="cuda")
    new, ctx = [3, 2], [45, 20]
    table = np.array([[pages - 1, 0, pages - 2], [pages - 40, 1, 2]])
    small = _case(new, ctx, hk, 1, dim, ps, "bf16")
    cache = sd.PagedCache(k, v)
    # store every key and value through the operator, then attend
    slots, ks, vs = [], [], []
    for l, s in enumerate(small["seq"]):
        for j in range(s):
            slots.append(int(table[l][j // ps]) * ps + j % ps)
            ks.append(small["k"][small["table"][l][j // ps], j % ps])
            vs.append(small["v"][small["table"][l][j // ps], j % ps])
    sd.spec_paged_store(torch.stack(ks), torch.stack(vs), torch.tensor(slots, device="cuda"), cache)
    big = dict(small, k=k, v=v, table=table)
    out, lse = _attend(sd, big)
    _check(small, out, lse)


def test_other_stream_and_graph(sd):
    import torch
    c = _case([8, 8], [300, 77], 2, 4, 128, 16, "bf16")
    cache = sd.PagedCache(c["k"], c["v"])
    batch = sd.PagedBatch(_i32(c["table"].tolist()), _i32(c["cu"]), _i32(c["seq"]), page_size=16)
    out, lse = torch.full_like(c["q"], 7.5), torch.full(c["q"].shape[:2], 7.5, device="cuda")
    ws = sd.new_attention_workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sd.spec_paged_attention(c["q"], cache, batch, 128 ** -0.5, out, lse, ws)
    s.synchronize()
    _check(c, out, lse)
    out.fill_(7.5)
    lse.fill_(7.5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sd.spec_paged_attention(c["q"], cache, batch, 128 ** -0.5, out, lse, ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    sd.spec_device_status()
    _check(c, out, lse)


def test_no_lse_and_nothing_to_do(sd):
    import torch
    c = _case([3], [20], 1, 2, 64, 16, "bf16")
    cache = sd.PagedCache(c["k"], c["v"])
    batch = sd.PagedBatch(_i32(c["table"].tolist()), _i32(c["cu"]), _i32(c["seq"]), page_size=16)
    out = torch.full_like(c["q"], 7.5)
    ws = sd.new_attention_workspace()
    sd.spec_paged_attention(c["q"], cache, batch, 0.125, out, None, ws)
    with_lse, lse = _attend(sd, c)
    assert torch.equal(out, with_lse)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    sd.spec_paged_attention(e, cache, batch, 0.125, e, None, ws)        # no tokens
    zero = _case([0, 0], [20, 0], 1, 2, 64, 16, "bf16")
    out, lse = _attend(sd, zero)                                         # lanes without tokens
    assert (out == 7.5).all() and (lse == 7.5).all()


# ---- a step ------------------------------------------------------------------

def test_plan_store_attend(sd):
    """Two steps of a small batch through all three calls, lengths on the device."""
    import torch
    lanes, ps, hk, group, dim = 3, 16, 2, 2, 64
    pages = 40
    k, v = (torch.full((pages, ps, hk, dim), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache, b = sd.PagedCache(k, v), sd.PagedBatch.create(lanes, 8, 80, ps)
    free = torch.randperm(pages, device="cuda").to(torch.int32)
    cursor = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = sd.new_attention_workspace()
    all_k, all_v = [[] for _ in range(lanes)], [[] for _ in range(lanes)]
    for step, new in enumerate(([20, 33, 1], [5, 1, 17])):
        b.new_lens.copy_(_i32(new))
        sd.spec_paged_plan(b, free, cursor)
        nk, nv = (torch.randn((80, hk, dim), device="cuda").to(torch.bfloat16) for _ in range(2))
        q = torch.randn((80, hk * group, dim), device="cuda").to(torch.bfloat16)
        sd.spec_paged_store(nk, nv, b.slots, cache)
        out, lse = sd.paged_attention(q, cache, b, workspace=ws)
        cu = b.cu_new.cpu().tolist()
        assert cu == [0] + np.cumsum(new).tolist()
        for l in range(lanes):
            all_k[l].append(nk[cu[l]:cu[l + 1]])
            all_v[l].append(nv[cu[l]:cu[l + 1]])
        # the reference reads plain per-lane keys: one page a lane
        longest = max(sum(x.shape[0] for x in a) for a in all_k)
        pk, pv = (torch.zeros((lanes, longest, hk, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for l in range(lanes):
            kk, vv = torch.cat(all_k[l]), torch.cat(all_v[l])
            pk[l, :kk.shape[0]], pv[l, :vv.shape[0]] = kk, vv
        c = dict(q=q, k=pk, v=pv, table=np.arange(lanes)[:, None], cu=cu, seq=b.seq_lens.cpu().tolist(), dtype="bf16", window=0)
        out[cu[-1]:], lse[cu[-1]:] = 7.5, 7.5
        _check(c, out, lse)
        # the next step starts where this one ended
        b.context_lens.copy_(b.seq_lens)
        b.held.copy_(b.held_out)
        cursor.copy_(b.info[1:2])
    assert b.info.cpu().tolist()[2:] == [0, 0]


# ---- further shapes, refusals with tensors, and an example -----------------------

def test_large_group_and_cut_queries(sd):
    """A group of more heads than a tile has rows; a query buffer shorter than
    the step, whose tokens keep their positions."""
    c = _case([2, 1], [30, 300], 1, 150, 64, 16, "bf16")
    out, lse = _attend(sd, c)
    _check(c, out, lse)
    c = _case([5, 8, 3], [30, 300, 10], 2, 2, 128, 16, "bf16")
    out, lse = _attend(sd, c, q=c["q"][:9].contiguous())
    whole_out, whole_lse = _attend(sd, c)
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    o, ls, ob, lb = ref.attention(f(c["q"]), f(c["k"]), f(c["v"]), c["table"], c["cu"], c["seq"], 128 ** -0.5, 0, "bf16")
    assert (np.abs(f(out) - o[:9]) <= ob[:9]).all() and (np.abs(f(lse) - ls[:9]) <= lb[:9]).all()


def test_lengths_that_are_none(sd):
    """Negative chunk boundaries and lengths past the table end the call all
    the same; other lanes are answered."""
    import torch
    c = _case([2, 3, 1], [30, 20, 40], 1, 2, 64, 16, "bf16")
    cache = sd.PagedCache(c["k"], c["v"])
    out, lse = torch.zeros_like(c["q"]), torch.zeros(c["q"].shape[:2], device="cuda")
    ws = sd.new_attention_workspace()
    b = sd.PagedBatch(_i32(c["table"].tolist()), _i32([0, 2, 1, 6]), _i32(c["seq"]), page_size=16)
    sd.spec_paged_attention(c["q"], cache, b, 0.125, out, lse, ws)
    seq = [c["seq"][0], 200, c["seq"][2]]      # past the lane's pages and the table: zero keys there
    b = sd.PagedBatch(_i32(c["table"].tolist()), _i32(c["cu"]), _i32(seq), page_size=16)
    sd.spec_paged_attention(c["q"], cache, b, 0.125, out, lse, ws)
    torch.cuda.synchronize()
    sd.spec_device_status()
    good, glse = _attend(sd, c)
    # (lane 1 attends what its last page holds past its keys: no promise is made for it)
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[5:6], good[5:6])


def test_two_streams_at_once(sd):
    """Calls that overlap, each with a workspace of its own."""
    import torch
    cases = [_case([3, 1], [9_000, 12_000], 2, 2, 128, 64, "bf16", seed=s) for s in (1, 2)]
    want = [_attend(sd, c) for c in cases]
    streams, got = [torch.cuda.Stream() for _ in cases], []
    for s, c in zip(streams, cases):
        s.wait_stream(torch.cuda.current_stream())
        cache = sd.PagedCache(c["k"], c["v"])
        b = sd.PagedBatch(_i32(c["table"].tolist()), _i32(c["cu"]), _i32(c["seq"]), page_size=64)
        got.append((cache, b, torch.full_like(c["q"], 7.5), torch.full(c["q"].shape[:2], 7.5, device="cuda"), sd.new_attention_workspace()))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, c, (cache, b, out, lse, ws) in zip(streams, cases, got):
            with torch.cuda.stream(s):
                sd.spec_paged_attention(c["q"], cache, b, 128 ** -0.5, out, lse, ws)
    torch.cuda.synchronize()
    sd.spec_device_status()
    for (wo, wl), (_, _, out, lse, _) in zip(want, got):
        assert torch.equal(out, wo) and torch.equal(lse, wl)


def test_binding_refuses(sd):
    import torch
    c = _case([2], [20], 2, 2, 64, 16, "bf16")
    cache = sd.PagedCache(c["k"], c["v"])
    b = sd.PagedBatch(_i32(c["table"].tolist()), _i32(c["cu"]), _i32(c["seq"]), page_size=16)
    q, ws = c["q"], sd.new_attention_workspace()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")

    def refused(text, f, *a, **k):
        with pytest.raises(sd.SpecError) as ei:
            f(*a, **k)
        assert ei.value.status == sd.SPEC_ERR_ARG and text in str(ei.value), str(ei.value)
    at = sd.spec_paged_attention
    refused("dtype", at, q.half(), cache, b, 0.1, out, lse, ws)
    refused("shape", at, q[:, :, :32], cache, b, 0.1, out, lse, ws)
    refused("contiguous", at, q.transpose(1, 2).contiguous().transpose(1, 2), cache, b, 0.1, out, lse, ws)
    refused("out", at, q, cache, b, 0.1, out[:1], lse, ws)
    refused("lse", at, q, cache, b, 0.1, out, lse.half(), ws)
    refused("workspace", at, q, cache, b, 0.1, out, lse, ws[:100])
    refused("heads_q", at, q[:, :3], cache, b, 0.1, torch.empty_like(q[:, :3]).contiguous(), lse, ws)
    refused("k:", sd.spec_paged_store, q[:, :1], q[:, :2], torch.zeros(9, dtype=torch.int64, device="cuda"), cache)
    refused("slots", sd.spec_paged_store, q[:, :2], q[:, 2:], torch.zeros(q.shape[0], dtype=torch.int32, device="cuda"), cache)
    refused("plan's buffers", sd.spec_paged_plan, b, _i32([1]))
    refused("last dimension", sd.PagedCache, c["k"].transpose(2, 3), c["v"].transpose(2, 3))
    refused("one shape", sd.PagedCache, c["k"], c["v"][:1])
    refused("go together", sd.PagedBatch, _i32(c["table"].tolist()), _i32(c["cu"]), _i32(c["seq"]), page_size=16, held=_i32([1]))
    x = torch.zeros((2, 50), dtype=torch.bfloat16, device="cuda")
    refused("dtype", sd.process_logits, x.float(), 2, 1)
    refused("penalties", sd.process_logits, x, 2, 1, penalties=torch.zeros((1, 3), device="cuda"))
    refused("mask", sd.process_logits, x, 2, 1, mask=_i32([[1]]), mask_rows=_i32([0, 0]))
    refused("go together", sd.process_logits, x, 2, 1, history=_i32([[1], [2]]))


def test_example_round(sd):
    """The example loop: every committed token is the argmax of its processed
    column, allowed by the grammar and said once; the cache holds the keys and
    values of exactly the tokens committed before the last anchor."""
    import importlib.util
    import os
    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_round.py")
    spec = importlib.util.spec_from_file_location("paged_round", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.generate(lanes=3, rounds=6, seed=4)
    torch.cuda.synchronize()
    sd.spec_device_status()
    toy, cache, batch = r["toy"], r["cache"], r["batch"]
    assert r["accepted"].shape == (6, 3) and int(r["accepted"].min()) >= 0 and int(r["accepted"].max()) <= 7
    assert int(r["accepted"].sum()) > 0, "the drafter is meant to be right sometimes"
    assert batch.info.cpu().tolist()[2:] == [0, 0]
    top = r["last_target"].float().argmax(1).view(3, 8)
    for lane in range(3):
        p, s = int(r["prompt"][lane]), int(r["said"][lane])
        said = r["history"][lane, p:s].long()
        assert s - p == int(r["accepted"][:, lane].sum()) + 6
        assert bool(toy.allowed[said].all()) and len(set(said.tolist())) == s - p
        a = int(r["accepted"][-1, lane])
        best = r["last_target"][lane * 8:lane * 8 + 8].float()
        committed = r["last_commits"][lane, :a + 1].long()
        assert torch.equal(best[torch.arange(a + 1), committed], best[torch.arange(a + 1), top[lane, :a + 1]])
        n = int(batch.context_lens[lane])
        assert n == s - 1                      # the last commit is the next anchor
        j = torch.arange(n, device="cuda")
        page = batch.block_table[lane].long()[j // cache.page_size]
        ids = r["history"][lane, :n].long()
        assert torch.equal(cache.k[page, j % cache.page_size], toy.k[ids]) and torch.equal(cache.v[page, j % cache.page_size], toy.v[ids])
