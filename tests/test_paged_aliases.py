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


# where each buffer of an attention call lies: 4 tokens of 6 heads of 64 (3,072 bytes), tables of 3 lanes
Q, OUT, LSE, TABLE, CU, SEQ, WS, WS_BYTES = 0x200000, 0x210000, 0x220000, 0x230000, 0x240000, 0x250000, 0x1000000, 1 << 40


def _attend(sd, q=Q, out=OUT, lse=LSE, table=TABLE, cu=CU, seq=SEQ, ws=WS, token_stride=6 * 64, head_stride=64, tokens=4):
    three = ctypes.c_int64 * 3
    c = sd.paged._CacheStruct(0x300000, 0x400000, three(2048, 128, 64), three(2048, 128, 64), 10, 16, 2, 64, sd.SPEC_BF16)
    b = sd.paged._BatchStruct(block_table=table, cu_new=cu, seq_lens=seq, lanes=3, max_pages=8, page_size=16)
    return sd.lib.spec_paged_attention(q, tokens, 6, token_stride, head_stride, ctypes.byref(c), ctypes.byref(b), 0.1, 0, 0, out,
                                       lse, ws, WS_BYTES)


@pytest.mark.parametrize("at", [-3_072 + 16, -16, 0, 16, 3_072 - 16])
def test_out_over_queries(sd, at):
    """Wherever out begins: before q's first element, at it, or among its rows."""
    _refused(sd, _attend(sd, out=Q + at), "out overlaps q")


def test_out_over_strided_queries(sd):
    """Queries whose rows lie apart: up to the last row's last element."""
    last = 3 * 18 * 64 + 5 * 64 + 64
    for at in (0, 6 * 64 * 2, (last - 8) * 2):
        _refused(sd, _attend(sd, out=Q + at, token_stride=18 * 64), "out overlaps q")
        _refused(sd, _attend(sd, lse=Q + at, token_stride=18 * 64), "lse overlaps q")
    # strides whose product is past 64 bits are no way round the check
    _refused(sd, _attend(sd, out=Q + (1 << 30), token_stride=(1 << 39) - 8, tokens=1 << 27), "out overlaps q")


@pytest.mark.parametrize("name,size", [("table", 3 * 8 * 4), ("cu", 16), ("seq", 12)])
def test_results_over_what_is_read(sd, name, size):
    at = dict(table=TABLE, cu=CU, seq=SEQ)[name]
    for where in (at, at + size - 4, at - 32):
        _refused(sd, _attend(sd, lse=where), "lse overlaps")
        _refused(sd, _attend(sd, out=where // 16 * 16), "out overlaps")


def test_results_over_each_other(sd):
    for at in (-92, 0, 3_072 - 4):
        _refused(sd, _attend(sd, lse=OUT + at), "out overlaps lse")
