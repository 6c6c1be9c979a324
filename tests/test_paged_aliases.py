"""Buffers of the paged-cache calls that overlap where one is read while the
other is written are refused, on the host (no GPU): every call below fails its
checks before any CUDA call."""
import ctypes
import os
import shutil

import pytest


@pytest.fixture(scope="module")
def sd():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    import __graft_entry__ as g
    g._load_build_module().build()
    import speculative_decoding_draft_column_gb300 as m
    return m


# where each buffer of a plan lies (never dereferenced): 4 lanes, 10 tokens, tables of 8 pages, 6 free pages
PLAN = dict(context_lens=0x100000, new_lens=0x101000, held=0x102000, block_table=0x103000, cu_new=0x104000, seq_lens=0x105000,
            held_out=0x106000, positions=0x107000, slots=0x108000, info=0x109000)
FREE, CURSOR = 0x10A000, 0x10B000
SIZE = dict(context_lens=16, new_lens=16, held=16, block_table=4 * 8 * 4, cu_new=20, seq_lens=16, held_out=16, positions=40,
            slots=80, info=16, free=24, cursor=4)


def _plan(sd, cursor=CURSOR, free=FREE, **kw):
    b = sd.paged._BatchStruct(lanes=4, max_pages=8, tokens=10, page_size=16, **dict(PLAN, **kw))
    return sd.lib.spec_paged_plan(ctypes.byref(b), free, 6, cursor)


def _refused(sd, st, *text):
    assert st == sd.SPEC_ERR_ARG and all(t in sd.spec_last_error() for t in text), (st, sd.spec_last_error())


@pytest.mark.parametrize("word", [0, 1, 2, 3])
def test_cursor_inside_info(sd, word):
    """info[1] is the next step's cursor: read by every CTA, written by the first."""
    _refused(sd, _plan(sd, cursor=PLAN["info"] + 4 * word), "alias", "info", "cursor")


@pytest.mark.parametrize("out", ["info", "held_out", "seq_lens", "cu_new", "positions", "slots", "block_table"])
@pytest.mark.parametrize("inp", ["context_lens", "new_lens", "held", "free", "cursor"])
def test_plan_outputs_over_inputs(sd, out, inp):
    """The output's first bytes over the input's last, and its last over the input's first."""
    at = {"free": FREE, "cursor": CURSOR}.get(inp, PLAN.get(inp))
    step = 8 if out == "slots" else 4
    for where in (at + SIZE[inp] - 4, at - SIZE[out] + step):
        where = where // step * step
        _refused(sd, _plan(sd, **{out: where}), "alias", out)
