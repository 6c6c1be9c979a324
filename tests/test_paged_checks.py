"""Refusals of the paged-cache and logits calls, on the host (no GPU): the C
checks fail before any CUDA call, the binding's before the library is called."""
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


P = 0x100000          # never dereferenced: every call below fails its checks first


def _cache(sd, **kw):
    three = ctypes.c_int64 * 3
    f = dict(k=P, v=P, k_strides=three(2048, 128, 64), v_strides=three(2048, 128, 64), pages=10, page_size=16, heads=2,
             head_dim=64, dtype=sd.SPEC_BF16)
    f.update({k: three(*v) if k.endswith("strides") else v for k, v in kw.items()})
    return sd.paged._CacheStruct(**f)


def _batch(sd, **kw):
    f = dict(context_lens=P, new_lens=P, held=P, block_table=P, cu_new=P, seq_lens=P + 64, held_out=P + 64, positions=P,
             slots=P, info=P, lanes=3, max_pages=8, tokens=20, page_size=16)
    f.update(kw)
    return sd.paged._BatchStruct(**f)


def _refused(sd, st, text):
    assert st == sd.SPEC_ERR_ARG and text in sd.spec_last_error(), (st, sd.spec_last_error())


@pytest.mark.parametrize("kw,text", [
    (dict(context_lens=None), "null"), (dict(slots=None), "null"), (dict(info=None), "null"), (dict(info=P + 2), "misaligned"),
    (dict(slots=P + 4), "slots need 8"), (dict(lanes=-1), "lanes"), (dict(lanes=4097), "lanes"), (dict(max_pages=0), "max_pages"),
    (dict(tokens=-1), "tokens"), (dict(page_size=0), "page_size"), (dict(held_out=P), "alias"), (dict(seq_lens=P), "alias")])
def test_plan_refusals(sd, kw, text):
    _refused(sd, sd.lib.spec_paged_plan(ctypes.byref(_batch(sd, **kw)), P, 5, None), text)


def test_plan_free_list_refusals(sd):
    b = _batch(sd)
    _refused(sd, sd.lib.spec_paged_plan(None, P, 5, None), "batch")
    _refused(sd, sd.lib.spec_paged_plan(ctypes.byref(b), None, 5, None), "null")
    _refused(sd, sd.lib.spec_paged_plan(ctypes.byref(b), P, -1, None), "num_free")
    _refused(sd, sd.lib.spec_paged_plan(ctypes.byref(b), P, 5, P + 1), "misaligned")


CACHE_REFUSALS = [
    (dict(k=None), "null"), (dict(v=P + 8), "16-byte"), (dict(dtype=7), "dtype"), (dict(pages=0), "pages"),
    (dict(heads=0), "heads"), (dict(head_dim=12), "head_dim"), (dict(head_dim=264), "head_dim"), (dict(page_size=0), "page_size"),
    (dict(k_strides=(2048, 129, 64)), "strides"), (dict(v_strides=(-2048, 128, 64)), "strides"),
    (dict(v_strides=(1 << 39, 128, 64)), "strides")]


@pytest.mark.parametrize("kw,text", CACHE_REFUSALS)
def test_cache_refusals(sd, kw, text):
    c, b = _cache(sd, **kw), _batch(sd)
    _refused(sd, sd.lib.spec_paged_store(P, P, 4, 128, 64, 128, 64, P, ctypes.byref(c)), text)
    _refused(sd, sd.lib.spec_paged_attention(P, 4, 4, 256, 64, ctypes.byref(c), ctypes.byref(b), 0.1, 0, 0, P, None, P, 1 << 40), text)


def test_store_refusals(sd):
    c = ctypes.byref(_cache(sd))
    f = sd.lib.spec_paged_store
    _refused(sd, f(P, P, -1, 128, 64, 128, 64, P, c), "tokens")
    _refused(sd, f(None, P, 4, 128, 64, 128, 64, P, c), "null")
    _refused(sd, f(P, P + 2, 4, 128, 64, 128, 64, P, c), "misaligned")
    _refused(sd, f(P, P, 4, 127, 64, 128, 64, P, c), "strides")
    _refused(sd, f(P, P, 4, 128, 64, 128, 64, P + 4, c), "misaligned")
    assert f(None, None, 0, 128, 64, 128, 64, None, c) == sd.SPEC_OK


def test_attention_refusals(sd):
    def call(q=P, tokens=4, heads=4, qt=256, qh=64, cache=None, batch=None, scale=0.1, window=0, max_new=0, out=P, lse=None,
             ws=P, wb=1 << 40):
        return sd.lib.spec_paged_attention(q, tokens, heads, qt, qh, ctypes.byref(cache or _cache(sd)),
                                           ctypes.byref(batch or _batch(sd)), scale, window, max_new, out, lse, ws, wb)
    _refused(sd, call(cache=_cache(sd, head_dim=96)), "64, 128 or 256")
    _refused(sd, call(cache=_cache(sd, page_size=24), batch=_batch(sd, page_size=24)), "powers of two")
    _refused(sd, call(cache=_cache(sd, page_size=4), batch=_batch(sd, page_size=4)), "powers of two")
    _refused(sd, call(batch=_batch(sd, page_size=32)), "differ")
    _refused(sd, call(heads=3), "heads_q")
    _refused(sd, call(heads=0), "heads_q")
    _refused(sd, call(tokens=-1), "tokens")
    _refused(sd, call(tokens=1 << 30), "2^31")
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        _refused(sd, call(scale=scale), "scale")
    _refused(sd, call(window=-1), "window")
    _refused(sd, call(max_new=-1), "max_new")
    _refused(sd, call(qt=255), "strides")
    _refused(sd, call(q=None), "null")
    _refused(sd, call(ws=None), "null")
    _refused(sd, call(q=P + 2), "misaligned")
    _refused(sd, call(out=P + 8), "misaligned")
    _refused(sd, call(lse=P + 1), "misaligned")
    _refused(sd, call(batch=_batch(sd, cu_new=None)), "null")
    assert call(tokens=0, q=None, out=None, ws=None) == sd.SPEC_OK
    assert call(batch=_batch(sd, lanes=0)) == sd.SPEC_OK


def test_attention_in_place_is_refused(sd):
    def call(q, out):
        return sd.lib.spec_paged_attention(q, 4, 4, 256, 64, ctypes.byref(_cache(sd)), ctypes.byref(_batch(sd)), 0.1, 0, 0, out,
                                           None, P, 1 << 40)
    _refused(sd, call(P, P), "overlaps")
    _refused(sd, call(P + 4 * 256 * 2 - 16, P), "overlaps")


def test_logits_refusals(sd):
    def call(lg=P, lanes=2, cols=3, V=100, h=None, hs=0, pl=None, hl=None, d=None, pen=None, bi=None, bv=None, nb=0, bl=None,
             m=None, mc=0, mr=None, out=P + (1 << 20)):
        return sd.lib.spec_logits_process(lg, lanes, cols, V, h, hs, pl, hl, d, pen, bi, bv, nb, bl, m, mc, mr, out)
    _refused(sd, call(lanes=-1), "lanes")
    _refused(sd, call(lanes=65_536), "lanes")
    _refused(sd, call(cols=0), "cols")
    _refused(sd, call(cols=17), "cols")
    _refused(sd, call(V=0), "V")
    _refused(sd, call(hs=-1), "negative")
    _refused(sd, call(lg=None), "null")
    _refused(sd, call(h=P, hs=4, pl=P), "go together")
    _refused(sd, call(bi=P, nb=4), "go together")
    _refused(sd, call(m=P, mc=1), "go together")
    _refused(sd, call(lg=P + 1), "misaligned")
    _refused(sd, call(pen=P + 2), "misaligned")
    _refused(sd, call(out=P + 2), "overlaps")
    assert call(lanes=0, lg=None, out=None) == sd.SPEC_OK
    assert sd.spec_launch_count() == 0


def test_binding_refusals(sd):
    import torch
    z = torch.zeros
    bf = lambda *n: z(n, dtype=torch.bfloat16)  # noqa: E731

    def refused(f, text):
        with pytest.raises(sd.SpecError) as ei:
            f()
        assert ei.value.status == sd.SPEC_ERR_ARG and text in str(ei.value), str(ei.value)
    refused(lambda: sd.PagedCache(bf(2, 16, 2, 64), bf(2, 16, 2, 64)), "CUDA")
    i32 = lambda *n: z(n, dtype=torch.int32)  # noqa: E731
    refused(lambda: sd.PagedBatch(i32(2, 4), i32(3), i32(2), page_size=16), "CUDA")
    refused(lambda: sd.PagedBatch(i32(8), i32(3), i32(2), page_size=16), "[lanes, max_pages]")
    if not torch.cuda.is_available():
        with pytest.raises(Exception):
            sd.spec_logits_process(bf(2, 10), 2, 1, 10, bf(2, 10))
