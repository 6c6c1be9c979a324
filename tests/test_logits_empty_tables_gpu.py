"""Logits rules with tables of no entries: a history of which nothing was said
yet, no biases, no grammar in use.  An empty tensor has no address; each is
the same as the rule left out.  Needs a GPU."""
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


def _tables(lanes, cols, V):
    """Each rule's tensors with no entries."""
    import torch
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return {
        "history": dict(history=i32(lanes, 0), prompt_lens=i32(lanes) + 3, history_lens=i32(lanes) + 5),
        "biases": dict(bias_ids=i32(lanes, 0), bias_vals=torch.zeros((lanes, 0), device="cuda"), bias_lens=i32(lanes) + 2),
        "mask": dict(mask=i32(0, (V + 31) // 32), mask_rows=i32(lanes * cols) - 1),
        "mask, rows past it": dict(mask=i32(0, (V + 31) // 32), mask_rows=i32(lanes * cols)),
    }


@pytest.mark.parametrize("rule", ["history", "biases", "mask", "mask, rows past it"])
def test_empty_table(sd, rule):
    import torch
    lanes, cols, V = 3, 2, 5_003
    x = torch.randn((lanes * cols, V), device="cuda").to(torch.bfloat16)
    drafts = torch.tensor([[7], [4_100], [5_002]], dtype=torch.int32, device="cuda")
    pen = torch.tensor([[1.3, 0.5, 0.25]] * lanes, device="cuda")
    want = sd.process_logits(x, lanes, cols, drafts=drafts, penalties=pen)
    assert not torch.equal(want, x)
    got = sd.process_logits(x, lanes, cols, drafts=drafts, penalties=pen, **_tables(lanes, cols, V)[rule])
    assert torch.equal(got, want)


def test_all_tables_empty(sd):
    import torch
    lanes, cols, V = 2, 3, 4_097
    x = torch.randn((lanes * cols, V), device="cuda").to(torch.bfloat16)
    rules = {}
    for r in _tables(lanes, cols, V).values():
        rules.update(r)
    assert torch.equal(sd.process_logits(x, lanes, cols, **rules), x)


def test_missing_tensors_are_still_refused(sd):
    """A rule of which a tensor is missing is no empty rule."""
    import torch
    x = torch.zeros((2, 50), dtype=torch.bfloat16, device="cuda")
    for rule in ("history", "biases", "mask"):
        whole = _tables(2, 1, 50)[rule]
        for name in whole:
            with pytest.raises(sd.SpecError) as ei:
                sd.process_logits(x, 2, 1, **{k: v for k, v in whole.items() if k != name})
            assert ei.value.status == sd.SPEC_ERR_ARG and "go together" in str(ei.value), str(ei.value)
