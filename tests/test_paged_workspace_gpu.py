"""What an attention call asks of its workspace: zeroed counters, and nothing
of the rest.  Needs a GPU."""
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


def _step(sd, new, ctx, hk, group, dim):
    import torch
    ps = 64
    pages = -(-(ctx + new) // ps)
    g = torch.Generator(device="cuda").manual_seed(dim + new)
    r = lambda *n: torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = sd.PagedBatch(torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1), i32([0, new]), i32([ctx + new]),
                          page_size=ps)
    return r(new, hk * group, dim), sd.PagedCache(r(pages, ps, hk, dim), r(pages, ps, hk, dim)), batch


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,ctx,hk,group", [(1, 5_000, 2, 4), (1, 30_000, 1, 3), (300, 3_000, 1, 2), (33, 0, 2, 4), (500, 100, 2, 1)])
def test_only_the_counters_are_zeroed(sd, dim, new, ctx, hk, group):
    """The parts' area holds NaN before the call; the counters are zero before and after it."""
    import torch
    q, cache, batch = _step(sd, new, ctx, hk, group, dim)
    want = sd.paged_attention(q, cache, batch, max_new=new, workspace=torch.zeros(
        sd.spec_paged_attention_workspace(), dtype=torch.uint8, device="cuda"))
    ws = torch.full((sd.spec_paged_attention_workspace(),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:sd.SPEC_PAGED_WORKSPACE_ZEROED] = 0
    for _ in range(2):
        out, lse = sd.paged_attention(q, cache, batch, max_new=new, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])
        assert not ws[:sd.SPEC_PAGED_WORKSPACE_ZEROED].any()
    sd.spec_device_status()


def test_new_workspace_clears_no_more(sd):
    """A workspace of some 40 MB is not cleared whole for a call of 10 us."""
    import torch
    dirty = torch.full((sd.spec_paged_attention_workspace(),), 0xFF, dtype=torch.uint8, device="cuda")
    at = dirty.data_ptr()
    torch.cuda.synchronize()
    del dirty                                             # (the allocator hands the same block out again)
    ws = sd.new_attention_workspace()
    assert ws.numel() == sd.spec_paged_attention_workspace()
    assert not ws[:sd.SPEC_PAGED_WORKSPACE_ZEROED].any()
    if ws.data_ptr() == at:
        assert bool((ws[sd.SPEC_PAGED_WORKSPACE_ZEROED:] == 0xFF).all())
