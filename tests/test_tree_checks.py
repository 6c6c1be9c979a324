"""Refusals of the tree and 8-bit cache calls, on the host (no GPU): the C checks
fail before any CUDA call, the binding's before the library is called."""
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
BIG = 1 << 40
THREE = ctypes.c_int64 * 3


def _cache8(sd, **kw):
    f = dict(k=P, v=P, k_scales=P, v_scales=P, k_strides=(2048, 128, 64), v_strides=(2048, 128, 64), pages=10, page_size=16,
             heads=2, head_dim=64, dtype=sd.SPEC_BF16)
    f.update(kw)
    return ctypes.byref(sd.paged._Cache8Struct(**{k: THREE(*v) if k.endswith("strides") else v for k, v in f.items()}))


def _cache(sd, **kw):
    f = dict(k=P, v=P, k_strides=(2048, 128, 64), v_strides=(2048, 128, 64), pages=10, page_size=16, heads=2, head_dim=64,
             dtype=sd.SPEC_BF16)
    f.update(kw)
    return ctypes.byref(sd.paged._CacheStruct(**{k: THREE(*v) if k.endswith("strides") else v for k, v in f.items()}))


def _batch(sd, **kw):
    f = dict(block_table=0x200000, cu_new=0x201000, seq_lens=0x202000, lanes=3, max_pages=8, tokens=20, page_size=16)
    f.update(kw)
    return ctypes.byref(sd.paged._BatchStruct(**f))


def _refused(sd, st, *text):
    assert st == sd.SPEC_ERR_ARG and all(t in sd.spec_last_error() for t in text), (st, sd.spec_last_error())


CACHE8 = [
    (dict(k=None), "null"), (dict(v_scales=None), "null"), (dict(k=P + 8), "16-byte"), (dict(k_scales=P + 4), "16-byte"),
    (dict(dtype=7), "dtype"), (dict(pages=0), "pages"), (dict(heads=0), "heads"), (dict(head_dim=24), "head_dim"),
    (dict(head_dim=272), "head_dim"), (dict(head_dim=0), "head_dim"), (dict(page_size=0), "page_size"),
    (dict(k_strides=(2048, 136, 64)), "multiples of 16"), (dict(v_strides=(-2048, 128, 64)), "strides"),
    (dict(v_strides=(1 << 39, 128, 64)), "strides"), (dict(heads=1 << 30), "heads * head_dim"),
    (dict(heads=1 << 24, page_size=1 << 30, pages=1 << 30), "too large")]


@pytest.mark.parametrize("kw,text", CACHE8)
def test_cache8_refusals(sd, kw, text):
    c, b = _cache8(sd, **kw), _batch(sd)
    _refused(sd, sd.lib.spec_paged_store8(P, P, 4, 128, 64, 128, 64, P, c), text)
    _refused(sd, sd.lib.spec_paged_attention8(P, 4, 4, 256, 64, c, b, 0.1, 0, 0, P, None, P, BIG), text)
    _refused(sd, sd.lib.spec_tree_attention8(P, 4, 4, 256, 64, c, b, P, 1, 0.1, 0, 0, P, None, P, BIG), text)
    _refused(sd, sd.lib.spec_tree_commit8(c, b, P, P, 3, P), text)


def test_store8_refusals(sd):
    c, f = _cache8(sd), sd.lib.spec_paged_store8
    _refused(sd, f(P, P, 4, 128, 64, 128, 64, P, None), "null")
    _refused(sd, f(P, P, -1, 128, 64, 128, 64, P, c), "tokens")
    _refused(sd, f(P, P, 1 << 31, 128, 64, 128, 64, P, c), "tokens")
    _refused(sd, f(None, P, 4, 128, 64, 128, 64, P, c), "null")
    _refused(sd, f(P, P + 2, 4, 128, 64, 128, 64, P, c), "misaligned")
    _refused(sd, f(P, P, 4, 128, 60, 128, 64, P, c), "strides")
    _refused(sd, f(P, P, 4, 128, 64, 128, 64, P + 4, c), "misaligned")
    assert f(None, None, 0, 128, 64, 128, 64, None, c) == sd.SPEC_OK


def test_attention8_refusals(sd):
    def call(cache=None, batch=None, heads=4, tokens=4, ws=P, out=P, q=P + (1 << 20)):
        return sd.lib.spec_paged_attention8(q, tokens, heads, 256, 64, cache or _cache8(sd), batch or _batch(sd), 0.1, 0, 0, out, None,
                                            ws, BIG)
    _refused(sd, call(cache=_cache8(sd, head_dim=48)), "64, 128 or 256")
    _refused(sd, call(cache=_cache8(sd, page_size=8), batch=_batch(sd, page_size=8)), "powers of two from 16")
    _refused(sd, call(cache=_cache8(sd, page_size=48), batch=_batch(sd, page_size=48)), "powers of two")
    _refused(sd, call(batch=_batch(sd, page_size=32)), "differ")
    _refused(sd, call(heads=3), "heads_q")
    _refused(sd, call(ws=None), "null")
    _refused(sd, call(out=P + 8), "misaligned")
    _refused(sd, call(q=P), "out overlaps q")
    assert call(tokens=0, ws=None, out=None, q=None) == sd.SPEC_OK


def test_few_rows_items_are_counted():
    """Items of 16 rows: where the host lets a step take them, they and their tiles fit the words they are counted in,
    lane by lane; the lanes need not have what the hint says."""
    import random
    rng = random.Random(7)
    for _ in range(2_000):
        lanes, hk, g = rng.randint(1, 60), rng.randint(1, 16), rng.randint(1, 16)
        new = [rng.choice([0, 1, 1, rng.randint(0, 900)]) for _ in range(lanes)]
        tokens = sum(new)
        bound = tokens * hk * g // 16 + min(tokens, lanes) * hk
        assert sum(-(-n * g // 16) for n in new) * hk <= bound
        if bound:
            most = ((1 << 40) // bound - 2) << 6              # keys of a lane at most
            assert bound * (-(-most // 64) + 1) < 1 << 40


def test_large_steps_with_a_small_hint_are_taken(sd):
    """2^26 items of 16 rows would not fit; items of 128 rows do."""
    c = _cache8(sd, heads=8, head_dim=128, k_strides=(1 << 20, 1024, 128), v_strides=(1 << 20, 1024, 128))
    st = sd.lib.spec_paged_attention8(P, 1 << 26, 8, 1024, 128, c, _batch(sd), 0.1, 0, 1, 1 << 44, None, None, 0)
    _refused(sd, st, "null pointer")


@pytest.mark.parametrize("eight", [False, True])
def test_tree_attention_refusals(sd, eight):
    f, cache = (sd.lib.spec_tree_attention8, _cache8(sd)) if eight else (sd.lib.spec_tree_attention, _cache(sd))

    def call(masks=0x300000, words=1, window=0, out=0x400000, lse=None, ws=0x1000000, batch=None):
        return f(P, 4, 4, 256, 64, cache, batch or _batch(sd), masks, words, 0.1, window, 0, out, lse, ws, BIG)
    _refused(sd, call(words=0), "mask_words")
    _refused(sd, call(words=9), "mask_words")
    _refused(sd, call(masks=None), "null")
    _refused(sd, call(masks=0x300002), "misaligned")
    _refused(sd, call(window=255), "window")
    _refused(sd, call(window=-1), "window")
    _refused(sd, call(masks=0x400000 + 16), "out overlaps masks")
    _refused(sd, call(lse=0x300004), "lse overlaps masks")
    _refused(sd, call(batch=_batch(sd, lanes=4097)), "lanes")


def test_plan_refusals(sd):
    def call(parents=0x300000, tokens=20, batch=None, masks=0x310000, words=2, positions=0x320000):
        return sd.lib.spec_tree_plan(parents, tokens, batch or _batch(sd), masks, words, positions)
    _refused(sd, sd.lib.spec_tree_plan(P, 4, None, P, 1, P), "batch")
    _refused(sd, call(tokens=-1), "tokens")
    _refused(sd, call(words=0), "mask_words")
    _refused(sd, call(words=9), "mask_words")
    _refused(sd, call(parents=None), "null")
    _refused(sd, call(positions=None), "null")
    _refused(sd, call(masks=0x310002), "misaligned")
    _refused(sd, call(masks=0x300000 + 76), "masks overlaps parents")
    _refused(sd, call(positions=0x201008), "positions overlaps cu_new")
    _refused(sd, call(masks=0x202004), "masks overlaps seq_lens")
    _refused(sd, call(positions=0x310000 + 4), "masks overlaps positions")
    assert call(tokens=0, parents=None, masks=None, positions=None) == sd.SPEC_OK
    assert call(batch=_batch(sd, lanes=0)) == sd.SPEC_OK


@pytest.mark.parametrize("sampled", [False, True])
def test_verify_refusals(sd, sampled):
    def call(logits=0x10000000, drafts=0x200000, parents=0x210000, cu=0x220000, tokens=20, lanes=3, depth=4, V=1_000, T=1.0, top_p=0.9,
             k=20, u=0x230000, acc=0x240000, com=0x250000, path=0x260000):
        if sampled:
            return sd.lib.spec_tree_verify_sampled(logits, drafts, parents, cu, tokens, lanes, depth, V, T, top_p, k, u, acc, com, path)
        return sd.lib.spec_tree_verify(logits, drafts, parents, cu, tokens, lanes, depth, V, acc, com, path)
    for kw, text in [(dict(lanes=-1), "lanes"), (dict(lanes=65_536), "lanes"), (dict(tokens=-1), "tokens"), (dict(depth=0), "depth"),
                     (dict(depth=256), "depth"), (dict(V=0), "V"), (dict(V=1 << 31), "V"), (dict(cu=None), "null"),
                     (dict(logits=None), "null"), (dict(path=None), "null"), (dict(logits=0x10000001), "misaligned"),
                     (dict(com=0x250002), "misaligned"), (dict(acc=0x200000 + 76), "out_accept_len overlaps drafts"),
                     (dict(com=0x10000000 + 39_996), "out_commit_ids overlaps target_logits"),
                     (dict(path=0x250000 + 56), "out_commit_ids overlaps out_path"), (dict(path=0x220000 + 12), "out_path overlaps cu"),
                     (dict(acc=0x260000 + 4), "overlaps")]:
        _refused(sd, call(**kw), text)
    if sampled:
        for kw, text in [(dict(T=0.0), "temperature"), (dict(T=float("inf")), "temperature"), (dict(top_p=0.0), "top_p"),
                         (dict(top_p=1.1), "top_p"), (dict(k=0), "top_k"), (dict(k=65), "top_k"), (dict(k=20, V=19), "top_k"),
                         (dict(u=None), "null"), (dict(u=0x230004), "misaligned"), (dict(acc=0x230000 + 8), "overlaps uniforms")]:
            _refused(sd, call(**kw), text)
    assert call(lanes=0, cu=None, logits=None) == sd.SPEC_OK


@pytest.mark.parametrize("eight", [False, True])
def test_commit_refusals(sd, eight):
    f, cache = (sd.lib.spec_tree_commit8, _cache8(sd)) if eight else (sd.lib.spec_tree_commit, _cache(sd))

    def call(batch=None, path=0x300000, acc=0x310000, depth=3, out=0x320000):
        return f(cache, batch or _batch(sd), path, acc, depth, out)
    _refused(sd, f(None, _batch(sd), P, P, 3, P), "null")
    _refused(sd, call(depth=0), "depth")
    _refused(sd, call(depth=256), "depth")
    _refused(sd, call(path=None), "null")
    _refused(sd, call(acc=0x310002), "misaligned")
    _refused(sd, call(batch=_batch(sd, page_size=32)), "differ")
    _refused(sd, call(batch=_batch(sd, seq_lens=None)), "null")
    for at, name in ((0x300000 + 44, "path"), (0x310000 - 8, "accept_lens"), (0x202000, "seq_lens"), (0x200000 + 92, "block_table"),
                     (0x201000 + 12, "cu_new")):
        _refused(sd, call(out=at), "context_out overlaps", name)
    assert call(batch=_batch(sd, lanes=0), path=None) == sd.SPEC_OK


def test_binding_refusals(sd):
    import torch
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(sd.SpecError) as ei:
        sd.PagedCache8(u8(2, 16, 2, 64), u8(2, 2, 16), u8(2, 16, 2, 64), u8(2, 2, 16))
    assert ei.value.status == sd.SPEC_ERR_ARG and "CUDA" in str(ei.value)
    for f in (sd.spec_paged_store, sd.spec_paged_store8):
        with pytest.raises(sd.SpecError) as ei:
            f(u8(1), u8(1), u8(1), object())
        assert "the call takes a PagedCache" in str(ei.value)
    for name in ("spec_tree_attention", "spec_tree_attention8", "spec_paged_attention8"):
        args = [u8(1, 1, 64), object(), None] + ([u8(1, 1)] if "tree" in name else []) + [0.1, None, None, None]
        with pytest.raises(sd.SpecError):
            getattr(sd, name)(*args)
    with pytest.raises(sd.SpecError):
        sd.spec_tree_commit(object(), None, None, None, 3)
    assert sd.spec_launch_count() == 0
