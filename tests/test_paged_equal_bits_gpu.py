"""Equal attention calls give equal bits, whichever CTA comes last at an item
that several share, and captured in a graph.  Needs a GPU."""
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


def _step(sd, new, ctx, hk, group, dim, ps, seed=0):
    """Cache, batch and queries of a step, pages in any order."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    seq = [c + n for c, n in zip(ctx, new)]
    need = [-(-s // ps) for s in seq]
    perm = torch.randperm(sum(need), generator=g, device="cuda").tolist()
    table = np.zeros((len(new), max(need)), dtype=np.int32)
    at = 0
    for lane, n in enumerate(need):
        table[lane, :n] = perm[at:at + n]
        at += n
    r = lambda *n: torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    cache = sd.PagedCache(r(sum(need), ps, hk, dim), r(sum(need), ps, hk, dim))
    batch = sd.PagedBatch(i32(table.tolist()), i32(np.concatenate([[0], np.cumsum(new)]).tolist()), i32(seq), page_size=ps)
    return r(sum(new), hk * group, dim), cache, batch


@pytest.mark.parametrize("cold", [False, True])
@pytest.mark.parametrize("dim,lanes,new,hk,group,tiles", [
    (64, 20, 1, 1, 8, 12), (64, 40, 8, 1, 4, 30), (64, 20, 4, 1, 4, 30), (128, 40, 1, 1, 8, 30), (128, 20, 1, 2, 4, 12),
    (128, 40, 4, 1, 4, 4), (128, 40, 8, 1, 4, 12), (256, 40, 1, 1, 8, 4), (256, 20, 1, 2, 4, 12),
    # narrower tables, for which the last CTA joins alone
    (64, 40, 8, 1, 4, 12), (64, 20, 4, 1, 4, 12), (64, 40, 4, 1, 4, 12), (128, 40, 1, 1, 8, 12)])
def test_ragged_lanes_repeat(sd, dim, lanes, new, hk, group, tiles, cold):
    """Lanes long and short in turn, whose items go to two to a dozen CTAs and
    are joined by the one that comes last: its other item has another number of
    parts, and which CTA it is, and whether it comes last at both, is timing."""
    import torch
    rng = np.random.default_rng(dim + lanes)
    keys = (64 if dim == 256 else 128) * 152 * tiles / (lanes * hk)          # `tiles` for each of 152 CTAs
    ctx = [int(keys * (1.5 if lane % 2 else 0.6) * rng.uniform(0.9, 1.1)) for lane in range(lanes)]
    q, cache, batch = _step(sd, [new] * lanes, ctx, hk, group, dim, 64, seed=1)
    ws = sd.new_attention_workspace()
    flush = torch.zeros(1 << 26, device="cuda") if cold else None
    want = [x.clone() for x in sd.paged_attention(q, cache, batch, max_new=new, workspace=ws)]
    differ, calls = 0, 100
    for _ in range(calls):
        if cold:
            flush.add_(1.0)
        out, lse = sd.paged_attention(q, cache, batch, max_new=new, workspace=ws)
        differ += not (torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1]))
    sd.spec_device_status()
    assert differ == 0, f"{differ} of {calls} equal calls gave other bits"


@pytest.mark.parametrize("dim,new,ctx,hk,group", [(128, [512, 300], [3_000, 900], 2, 4), (64, [1, 700], [9_000, 100], 1, 8),
                                                  (256, [128], [20_000], 1, 4)])
def test_shared_joins_in_a_graph(sd, dim, new, ctx, hk, group):
    """Large parts, whose CTAs join them together (a cooperative launch): a
    captured call, replayed, gives the bits of a plain one."""
    import torch
    q, cache, batch = _step(sd, new, ctx, hk, group, dim, 64)
    ws = sd.new_attention_workspace()
    want = sd.paged_attention(q, cache, batch, max_new=max(new), workspace=ws)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            sd.spec_paged_attention(q, cache, batch, dim ** -0.5, out, lse, ws, max_new=max(new))
    for _ in range(5):
        out.fill_(7.5)
        lse.fill_(7.5)
        graph.replay()
        torch.cuda.synchronize()
        sd.spec_device_status()
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])


@pytest.mark.parametrize("window", [1 << 20, 1 << 40, (1 << 63) - 1])
def test_a_window_past_every_key(sd, window):
    """Any window is taken; one wider than the context is none."""
    import torch
    for new, ctx, hk, group, dim in (([1, 3], [700, 20_000], 1, 4, 128), ([300], [2_000], 2, 4, 64)):
        q, cache, batch = _step(sd, new, ctx, hk, group, dim, 64)
        want = sd.paged_attention(q, cache, batch, max_new=max(new))
        out, lse = sd.paged_attention(q, cache, batch, max_new=max(new), window=window)
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_the_widest_window_over_rows_with_no_key(sd, dim):
    """A seq_len below the chunk: its first rows' positions lie below zero."""
    import torch
    for new, ctx, seq in (([4, 3], [0, 0], [2, 0]), ([200, 1], [0, 0], [150, 0])):
        q, cache, batch = _step(sd, new, ctx, 1, 4, dim, 64)
        batch.seq_lens.copy_(torch.tensor(seq, dtype=torch.int32))
        want = sd.paged_attention(q, cache, batch, max_new=max(new))
        assert (want[0][:new[0] - seq[0]] == 0).all() and want[1][:new[0] - seq[0]].isneginf().all()
        for window in (1 << 31, (1 << 63) - 1):
            out, lse = sd.paged_attention(q, cache, batch, max_new=max(new), window=window)
            assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])
