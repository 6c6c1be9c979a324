"""Attention of a batch with lanes that have no tokens, as fixed-size batches
in a graph have: its time is that of the lane that has some.  Needs a GPU."""
from __future__ import annotations

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


def _time(f, calls=10):
    """us of a call in a captured graph, the best of several replays."""
    import torch
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            f()
    best = float("inf")
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / calls)
    return best


@pytest.mark.parametrize("rest", [0, 1])
@pytest.mark.parametrize("dim,keys", [(128, 131_072), (64, 200_000)])
def test_one_long_lane_among_many(sd, dim, keys, rest):
    """One lane holds the keys of 64; the others have no tokens, or one token
    with one key.  Its item goes to all CTAs, and joining what they leave must
    not take longer than the attention itself: at most 8 us more than the lane
    by itself takes, where one CTA joining all its parts alone took 30 and more."""
    import torch
    lanes, new, group, ps = 64, 16, 4, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = -(-keys // ps)
    k, v = (torch.randn((pages + 1, ps, 1, dim), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((lanes * new, group, dim), generator=g, device="cuda").to(torch.bfloat16)
    cache, ws = sd.PagedCache(k, v), sd.new_attention_workspace()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    table = torch.full((lanes, pages), pages, dtype=torch.int32, device="cuda")
    table[0] = torch.arange(pages, dtype=torch.int32, device="cuda")
    alone = sd.PagedBatch(table[:1].contiguous(), i32([0, new]), i32([keys]), page_size=ps)
    many = sd.PagedBatch(table, i32([0] + [new + rest * i for i in range(lanes)]), i32([keys] + [rest] * (lanes - 1)), page_size=ps)
    run = lambda b, n: sd.spec_paged_attention(q[:n], cache, b, dim ** -0.5, out[:n], lse[:n], ws, max_new=new)  # noqa: E731
    run(alone, new)
    want = out[:new].clone()
    t_alone = _time(lambda: run(alone, new))
    run(many, lanes * new)
    # (the other lanes' items may cut the long one elsewhere: other roundings)
    assert (out[:new].float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()
    t_many = _time(lambda: run(many, lanes * new))
    sd.spec_device_status()
    assert t_many <= t_alone + 8.0, f"{t_many:.1f} us among {lanes} lanes, {t_alone:.1f} us by itself"
