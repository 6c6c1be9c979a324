"""Sizes that the paged-cache calls cannot count are refused, on the host (no
GPU): every call below fails its checks before any CUDA call."""
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


P = 0x100000          # never dereferenced


def _cache(sd, heads, head_dim=64):
    three = ctypes.c_int64 * 3
    return sd.paged._CacheStruct(P, P, three(2048, 128, 64), three(2048, 128, 64), 10, 16, heads, head_dim, sd.SPEC_BF16)


def _attend(sd, tokens, heads_q, heads, lanes):
    """A call without a workspace: of good sizes it is refused for that alone."""
    batch = sd.paged._BatchStruct(block_table=P, cu_new=P, seq_lens=P, lanes=lanes, max_pages=8, page_size=16)
    st = sd.lib.spec_paged_attention(P, tokens, heads_q, 64, 64, ctypes.byref(_cache(sd, heads)), ctypes.byref(batch), 0.1, 0, 0,
                                     P, None, None, 0)
    assert st == sd.SPEC_ERR_ARG
    return sd.spec_last_error()


@pytest.mark.parametrize("tokens,heads_q,heads,lanes", [
    (4_096, 2_048, 2_048, 4_096),          # an item for each lane and head: 2^23 and more
    (4_096, 4_096, 2_048, 4_096), (1 << 20, 2_047, 2_047, 4_096), (1 << 30, 1, 1, 1), (4, 1 << 28, 1 << 28, 4_096),
    (3, 1 << 23, 1 << 23, 1)])
def test_steps_of_too_many_items(sd, tokens, heads_q, heads, lanes):
    assert "row tiles" in _attend(sd, tokens, heads_q, heads, lanes) or "2^31" in _attend(sd, tokens, heads_q, heads, lanes)


@pytest.mark.parametrize("tokens,heads_q,heads,lanes", [
    (4_096, 2_000, 2_000, 4_096), (4, 2_048, 2_048, 4_096), (1_000_000, 64, 8, 64), ((1 << 30) - 256, 1, 1, 1), (262_144, 128, 8, 4_096)])
def test_large_steps_are_taken(sd, tokens, heads_q, heads, lanes):
    assert "null pointer" in _attend(sd, tokens, heads_q, heads, lanes)


def test_plan_of_the_runs_cannot_overflow():
    """The bound that the host checks, against a count of the items lane by
    lane; and tiles below 2^40 for whatever lengths the device holds."""
    import random
    rng = random.Random(5)
    for _ in range(2_000):
        lanes, hk, g = rng.randint(1, 40), rng.randint(1, 16), rng.randint(1, 150)
        new = [rng.choice([0, 1, 1, rng.randint(0, 700)]) for _ in range(lanes)]
        tokens = sum(new)
        items = sum(-(-n * g // 128) * hk for n in new)
        bound = tokens * hk * g // 128 + min(tokens, lanes) * hk
        assert items <= bound
        if bound:
            tiles = min(0x7FFF0000 >> 6, (1 << 40) // bound - 2)
            keys = tiles << 6
            assert items * (keys // 64 + 1) < 1 << 40
    for bound in (1, 1 << 14, 1 << 15, (1 << 23) - 1):
        tiles = min(0x7FFF0000 >> 6, (1 << 40) // bound - 2)
        assert tiles >= 1 << 16 and bound * (tiles + 1) < 1 << 40


def test_cache_rows_of_too_many_elements(sd):
    for heads, dim in ((1 << 28, 8), (1 << 25, 64), ((1 << 31) - 1, 256)):
        c = ctypes.byref(_cache(sd, heads, dim))
        assert sd.lib.spec_paged_store(P, P, 4, 128, 64, 128, 64, P, c) == sd.SPEC_ERR_ARG
        assert "heads * head_dim" in sd.spec_last_error()
    assert sd.lib.spec_paged_store(P, P, 4, 128, 64, 128, 64, None, ctypes.byref(_cache(sd, (1 << 25) - 1))) == sd.SPEC_ERR_ARG
    assert "null pointer" in sd.spec_last_error()
