"""Attention results in memory that the call uses otherwise.  Needs a GPU; the
refused calls launch nothing."""
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


def test_results_in_the_workspace_buffer(sd):
    """Inside what the call uses of the buffer: refused.  Past that: taken."""
    import torch
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    r = lambda *n: torch.randn(n, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, cache = r(5, 4, 64), sd.PagedCache(r(4, 16, 2, 64), r(4, 16, 2, 64))
    batch = sd.PagedBatch(i32([[2, 0, 1, 3]]), i32([0, 5]), i32([50]), page_size=16)
    need = sd.spec_paged_attention_workspace()
    ws = torch.zeros(need + 8_192, dtype=torch.uint8, device="cuda")
    want, lse = sd.paged_attention(q, cache, batch)
    launches = sd.spec_launch_count()
    for at in (0, 4_096, need - 16):
        for o, l in ((ws[at:at + 2_560].view(torch.bfloat16).view(5, 4, 64), lse),
                     (torch.empty_like(q), ws[at:at + 80].view(torch.float32).view(5, 4))):
            with pytest.raises(sd.SpecError) as ei:
                sd.spec_paged_attention(q, cache, batch, 0.125, o, l, ws)
            assert "workspace" in str(ei.value)
    assert sd.spec_launch_count() == launches
    at = -(-need // 16) * 16
    out = ws[at:at + 2_560].view(torch.bfloat16).view(5, 4, 64)
    sd.spec_paged_attention(q, cache, batch, 0.125, out, lse, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
