"""Binding of the paged cache (16 and 8 bits), the rounds of trees and the logits rules (see ``include/specsel.h``).

``PagedCache`` and ``PagedBatch`` describe a caller's tensors to the library:
they check them once, keep them alive and hold the C struct; they own no data
of their own unless made with ``create``.  The calls check what changes from
call to call, set the library's stream to PyTorch's current one and forward to
the C entry point of the same name.
"""
from __future__ import annotations

import ctypes

from . import SPEC_ERR_ARG, SpecError, _check, _n, lib

SPEC_BF16, SPEC_F16 = 0, 1
SPEC_PAGED_MAX_LANES, SPEC_PAGED_WORKSPACE_ZEROED = 4096, 4096
SPEC_TREE_MAX_NODES = 256

_p, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_strides", _i64 * 3), ("v_strides", _i64 * 3), ("pages", _i64),
                ("page_size", _i32), ("heads", _i32), ("head_dim", _i32), ("dtype", _i32)]


class _Cache8Struct(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_scales", _p), ("v_scales", _p), ("k_strides", _i64 * 3), ("v_strides", _i64 * 3),
                ("pages", _i64), ("page_size", _i32), ("heads", _i32), ("head_dim", _i32), ("dtype", _i32)]


class _BatchStruct(ctypes.Structure):
    _fields_ = [("context_lens", _p), ("new_lens", _p), ("held", _p), ("block_table", _p), ("cu_new", _p),
                ("seq_lens", _p), ("held_out", _p), ("positions", _p), ("slots", _p), ("info", _p),
                ("lanes", _i64), ("max_pages", _i64), ("tokens", _i64), ("page_size", _i32)]


def _bad(message):
    raise SpecError(SPEC_ERR_ARG, message)


def _dtype_code(x, name):
    import torch
    if x.dtype == torch.bfloat16:
        return SPEC_BF16
    if x.dtype == torch.float16:
        return SPEC_F16
    _bad(f"{name}: dtype {x.dtype}, need bfloat16 or float16")


def _load_torch():
    import torch
    global _torch, _raw_stream
    _torch = lambda: torch  # noqa: E731 - no import statement on the way of each call
    # the current stream's handle; the Stream object costs ten times as much
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    return torch


def _torch():
    return _load_torch()


def _raw_stream(dev):
    _load_torch()
    return _raw_stream(dev)


def _set_stream(dev):
    lib.spec_set_stream(_raw_stream(dev))


def _array(x, dtype, count, dev, name):
    """Pointer of a contiguous CUDA tensor of `dtype` on device `dev` with at
    least `count` elements; these calls take no raw pointers."""
    try:
        if x.dtype is dtype and x.get_device() == dev and x.numel() >= count and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        _bad(f"{name}: need a CUDA tensor")
    if x.get_device() != dev:
        _bad(f"{name}: on {x.device}, need cuda:{dev}")
    if x.dtype is not dtype:
        _bad(f"{name}: dtype {x.dtype}, need {dtype}")
    if not x.is_contiguous():
        _bad(f"{name}: tensor must be contiguous")
    _bad(f"{name}: {x.numel()} elements, the call needs {count}")


def _rows(x, shape, cache, name):
    """Strides of a [tokens, heads, head_dim] tensor of the cache's type and
    device whose rows are contiguous."""
    try:
        have, strides = x.shape, x.stride()
        if x.dtype is cache.torch_dtype and x.get_device() == cache.device and len(have) == 3 and strides[2] == 1 \
                and have[2] == cache.head_dim and (shape is None or have == shape):
            return strides
    except AttributeError:
        _bad(f"{name}: need a CUDA tensor on cuda:{cache.device}, where the cache is")
    if x.get_device() != cache.device:
        _bad(f"{name}: on {x.device}, the cache is on cuda:{cache.device}")
    if x.dtype is not cache.torch_dtype:
        _bad(f"{name}: dtype {x.dtype}, the cache's is {cache.torch_dtype}")
    if len(have) != 3 or have[2] != cache.head_dim or (shape is not None and have != shape):
        _bad(f"{name}: shape {tuple(have)}, need {shape or ('tokens', 'heads', cache.head_dim)}")
    if x.numel():
        _bad(f"{name}: the last dimension must be contiguous")
    return strides


def _rows_of(x, lanes, name):
    """Length of the rows of a [lanes, length] tensor."""
    shape = x.shape
    if len(shape) != 2 or shape[0] < lanes:
        _bad(f"{name}: need [lanes, length], got {tuple(shape)}")
    return shape[1]


def _is_cache(cache, kind):
    if type(cache) is not kind and not isinstance(cache, kind):
        _bad(f"cache: a {type(cache).__name__}, the call takes a {kind.__name__}")


def _on_current_device(index, name):
    cur = _torch().cuda.current_device()
    if index != cur:
        _bad(f"{name}: on cuda:{index}, the current device is cuda:{cur}")
    return cur


class PagedCache:
    """Keys and values of one layer: two CUDA tensors [pages, page_size, heads,
    head_dim], bf16 or fp16, each with any strides over the first three
    dimensions (a permuted view of [pages, heads, page_size, head_dim] serves)."""

    def __init__(self, k, v):
        for x, name in ((k, "k"), (v, "v")):
            if not getattr(x, "is_cuda", False):
                _bad(f"{name}: need a CUDA tensor")
            if x.dim() != 4:
                _bad(f"{name}: need [pages, page_size, heads, head_dim], got {tuple(x.shape)}")
            if x.stride(3) != 1:
                _bad(f"{name}: the last dimension must be contiguous")
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            _bad("k and v must have one shape, dtype and device")
        self.k, self.v = k, v
        self.pages, self.page_size, self.heads, self.head_dim = k.shape
        self.device, self.torch_dtype = k.device.index, k.dtype
        three = _i64 * 3
        self._c = _CacheStruct(k.data_ptr(), v.data_ptr(), three(*k.stride()[:3]), three(*v.stride()[:3]), self.pages,
                               self.page_size, self.heads, self.head_dim, _dtype_code(k, "k"))
        self._ref = ctypes.byref(self._c)


class PagedCache8:
    """Keys and values of one layer in 8 bits: codes in two CUDA tensors [pages, page_size, heads,
    head_dim] (torch.float8_e4m3fn, or uint8 with the same bits), any strides over the first three
    dimensions, and their scales in two contiguous uint8 tensors [pages, heads, page_size].  ``dtype``
    (torch.bfloat16 or torch.float16) is what is stored from and attended with.  Codes that are NaN
    need a scale above 134 (``spec_paged_store8`` writes 255)."""

    def __init__(self, k, k_scales, v, v_scales, *, dtype=None):
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        for x, name in ((k, "k"), (v, "v")):
            if not getattr(x, "is_cuda", False):
                _bad(f"{name}: need a CUDA tensor")
            if x.dtype not in (torch.float8_e4m3fn, torch.uint8):
                _bad(f"{name}: dtype {x.dtype}, need float8_e4m3fn or uint8")
            if x.dim() != 4:
                _bad(f"{name}: need [pages, page_size, heads, head_dim], got {tuple(x.shape)}")
            if x.stride(3) != 1:
                _bad(f"{name}: the last dimension must be contiguous")
        if k.shape != v.shape or k.device != v.device:
            _bad("k and v must have one shape and device")
        self.pages, self.page_size, self.heads, self.head_dim = k.shape
        self.device, self.torch_dtype = k.device.index, dtype
        for x, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _array(x, torch.uint8, self.pages * self.heads * self.page_size, self.device, name)
            if tuple(x.shape) != (self.pages, self.heads, self.page_size):
                _bad(f"{name}: shape {tuple(x.shape)}, need [pages, heads, page_size]")
        if dtype not in (torch.bfloat16, torch.float16):
            _bad(f"dtype {dtype}: need bfloat16 or float16")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        three = _i64 * 3
        self._c = _Cache8Struct(k.data_ptr(), v.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                three(*k.stride()[:3]), three(*v.stride()[:3]), self.pages, self.page_size, self.heads,
                                self.head_dim, SPEC_BF16 if dtype is torch.bfloat16 else SPEC_F16)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def create(cls, pages, page_size, heads, head_dim, dtype=None, device="cuda"):
        """A cache of its own zeroed codes and scales."""
        import torch
        z = lambda *n: torch.zeros(n, dtype=torch.uint8, device=device)  # noqa: E731
        shape, scales = (pages, page_size, heads, head_dim), (pages, heads, page_size)
        return cls(z(*shape), z(*scales), z(*shape), z(*scales), dtype=dtype)


class PagedBatch:
    """The lanes of a step: block_table int32 [lanes, max_pages], cu_new int32
    [lanes+1] and seq_lens int32 [lanes] for attention; the other buffers for
    spec_paged_plan (all or none)."""

    _PLAN = ("context_lens", "new_lens", "held", "held_out", "positions", "slots", "info")

    def __init__(self, block_table, cu_new, seq_lens, *, page_size, context_lens=None, new_lens=None, held=None,
                 held_out=None, positions=None, slots=None, info=None):
        import torch
        if block_table.dim() != 2:
            _bad("block_table: need [lanes, max_pages]")
        lanes, max_pages = block_table.shape
        self.lanes, self.max_pages, self.page_size = lanes, max_pages, page_size
        self.block_table, self.cu_new, self.seq_lens = block_table, cu_new, seq_lens
        i32, dev = torch.int32, block_table.get_device()
        if dev < 0:
            _bad("block_table: need a CUDA tensor")
        s = _BatchStruct(block_table=_array(block_table, i32, lanes * max_pages, dev, "block_table"),
                         cu_new=_array(cu_new, i32, lanes + 1, dev, "cu_new"),
                         seq_lens=_array(seq_lens, i32, lanes, dev, "seq_lens"),
                         lanes=lanes, max_pages=max_pages, page_size=page_size)
        self.device = dev
        rest = (context_lens, new_lens, held, held_out, positions, slots, info)
        self.plannable = all(x is not None for x in rest)
        if not self.plannable and any(x is not None for x in rest):
            _bad("the plan's buffers go together: " + ", ".join(self._PLAN))
        for name, x in zip(self._PLAN, rest):
            setattr(self, name, x)
        if self.plannable:
            tokens = positions.numel()
            for name, count in (("context_lens", lanes), ("new_lens", lanes), ("held", lanes), ("held_out", lanes),
                                ("positions", tokens), ("info", 4)):
                setattr(s, name, _array(getattr(self, name), i32, count, dev, name))
            s.slots = _array(slots, torch.int64, tokens, dev, "slots")
            s.tokens = tokens
        self._c = s
        self._ref = ctypes.byref(s)

    @classmethod
    def create(cls, lanes, max_pages, tokens, page_size, device="cuda"):
        """A batch of its own zeroed buffers, for up to `tokens` new tokens a step."""
        import torch
        z = lambda *n, dtype=torch.int32: torch.zeros(n, dtype=dtype, device=device)  # noqa: E731
        return cls(z(lanes, max_pages), z(lanes + 1), z(lanes), page_size=page_size, context_lens=z(lanes),
                   new_lens=z(lanes), held=z(lanes), held_out=z(lanes), positions=z(tokens),
                   slots=z(tokens, dtype=torch.int64), info=z(4))


def spec_paged_plan(batch, free_pages, cursor=None):
    """Plan a step into the batch's buffers; ``free_pages`` int32, ``cursor``
    int32 [1] (the pages of the list used before) or None.  The call writes the
    next step's cursor to ``batch.info[1]``: copy it from there, since a cursor
    inside ``info`` would be written while it is read, and is refused."""
    if not batch.plannable:
        _bad("batch: made without the plan's buffers")
    i32 = _torch().int32
    dev = _on_current_device(batch.device, "batch")
    n = free_pages.numel()
    f = _array(free_pages, i32, n, dev, "free_pages")
    c = None if cursor is None else _array(cursor, i32, 1, dev, "cursor")
    _set_stream(dev)
    st = lib.spec_paged_plan(batch._ref, f, n, c)
    if st:
        _check(st)


def _store(call, kind, k, v, slots, cache):
    _is_cache(cache, kind)
    tokens = k.shape[0]
    shape = (tokens, cache.heads, cache.head_dim)
    ks, vs = _rows(k, shape, cache, "k"), _rows(v, shape, cache, "v")
    dev = _on_current_device(cache.device, "cache")
    sl = _array(slots, _torch().int64, tokens, dev, "slots")
    _set_stream(dev)
    st = call(k.data_ptr(), v.data_ptr(), tokens, ks[0], ks[1], vs[0], vs[1], sl, cache._ref)
    if st:
        _check(st)


def spec_paged_store(k, v, slots, cache):
    """Store k, v [tokens, heads, head_dim] at slots int64 [tokens] of the cache."""
    _store(lib.spec_paged_store, PagedCache, k, v, slots, cache)


def spec_paged_store8(k, v, slots, cache):
    """The same into a PagedCache8, quantised: a power-of-two scale a vector, e4m3 codes."""
    _store(lib.spec_paged_store8, PagedCache8, k, v, slots, cache)


def spec_paged_attention_workspace() -> int:
    """Bytes of workspace an attention call needs on the current device."""
    n = int(lib.spec_paged_attention_workspace())
    if n < 0:
        _check(n)
    return n


def new_attention_workspace(device="cuda"):
    """A workspace for spec_paged_attention (one per stream that may run it), its counters zeroed."""
    import torch
    with torch.cuda.device(device):
        ws = torch.empty(spec_paged_attention_workspace(), dtype=torch.uint8, device=device)
        ws[:SPEC_PAGED_WORKSPACE_ZEROED].zero_()
        return ws


def _attention(call, kind, q, cache, batch, tree, scale, out, lse, workspace, window, max_new):
    _is_cache(cache, kind)
    shape = q.shape
    qs = _rows(q, None, cache, "q")
    dev = _on_current_device(cache.device, "cache")
    if batch.device != dev:
        _bad("batch and cache are on different devices")
    tokens, heads_q, dim = shape
    if out.shape != shape:
        _bad(f"out: shape {tuple(out.shape)}, need {tuple(shape)}")
    o = _array(out, cache.torch_dtype, tokens * heads_q * dim, dev, "out")
    ls = None if lse is None else _array(lse, _torch().float32, tokens * heads_q, dev, "lse")
    ws = _array(workspace, workspace.dtype, 0, dev, "workspace")
    if tree is not None:
        if tree.dim() != 2 or tree.shape[0] < tokens:
            _bad(f"masks: need [tokens, words], got {tuple(tree.shape)}")
        words = tree.shape[1]
        tree = (_array(tree, _torch().int32, tokens * words, dev, "masks"), words)
    _set_stream(dev)
    st = call(q.data_ptr(), tokens, heads_q, qs[0], qs[1], cache._ref, batch._ref, *(tree or ()), scale, window,
              max_new, o, ls, ws, workspace.numel() * workspace.element_size())
    if st:
        _check(st)


def spec_paged_attention(q, cache, batch, scale, out, lse, workspace, window=0, max_new=0):
    """Attention of the batch's new tokens: q [tokens, heads_q, head_dim] into
    out (same shape, contiguous) and lse fp32 [tokens, heads_q] (or None)."""
    _attention(lib.spec_paged_attention, PagedCache, q, cache, batch, None, scale, out, lse, workspace, window, max_new)


def spec_paged_attention8(q, cache, batch, scale, out, lse, workspace, window=0, max_new=0):
    """The same over a PagedCache8."""
    _attention(lib.spec_paged_attention8, PagedCache8, q, cache, batch, None, scale, out, lse, workspace, window, max_new)


def spec_tree_attention(q, cache, batch, masks, scale, out, lse, workspace, window=0, max_new=0):
    """Attention where a lane's new tokens are the nodes of a tree: masks int32 [tokens, words], bit b of word w
    set where the token sees its lane's new token 32 w + b (``spec_tree_plan`` writes them)."""
    _attention(lib.spec_tree_attention, PagedCache, q, cache, batch, masks, scale, out, lse, workspace, window, max_new)


def spec_tree_attention8(q, cache, batch, masks, scale, out, lse, workspace, window=0, max_new=0):
    """The same over a PagedCache8."""
    _attention(lib.spec_tree_attention8, PagedCache8, q, cache, batch, masks, scale, out, lse, workspace, window, max_new)


def spec_tree_plan(parents, batch, masks, positions):
    """Masks int32 [tokens, words] and positions int32 [tokens] of the step's trees, from parents int32 [tokens]."""
    t = _torch()
    dev = _on_current_device(batch.device, "batch")
    tokens = parents.numel()
    if masks.dim() != 2 or masks.shape[0] != tokens:
        _bad(f"masks: need [{tokens}, words], got {tuple(masks.shape)}")
    words = masks.shape[1]
    p, m = _array(parents, t.int32, tokens, dev, "parents"), _array(masks, t.int32, tokens * words, dev, "masks")
    at = _array(positions, t.int32, tokens, dev, "positions")
    _set_stream(dev)
    st = lib.spec_tree_plan(p, tokens, batch._ref, m, words, at)
    if st:
        _check(st)


def _tree_arrays(logits, drafts, parents, cu, lanes, depth, V, accept, commit, path):
    t = _torch()
    dev = t.cuda.current_device()
    if logits.dtype is not t.bfloat16 and logits.dtype not in (t.int16, t.uint16):
        _bad(f"target_logits: dtype {logits.dtype} is not bf16 bits")
    tokens, ln, width = drafts.numel(), _n(lanes), _n(depth) + 1
    i32 = t.int32
    return (dev, tokens, (_array(logits, logits.dtype, tokens * _n(V), dev, "target_logits"), _array(drafts, i32, tokens, dev, "drafts"),
                          _array(parents, i32, tokens, dev, "parents"), _array(cu, i32, ln + 1, dev, "cu")),
            (_array(accept, i32, ln, dev, "out_accept_len"), _array(commit, i32, ln * width, dev, "out_commit_ids"),
             _array(path, i32, ln * width, dev, "out_path")))


def spec_tree_verify(target_logits, drafts, parents, cu, lanes, depth, V, out_accept_len, out_commit_ids, out_path):
    """Greedy verify of trees: bf16 target_logits [tokens, V], drafts and parents int32 [tokens], cu int32 [lanes+1]
    into int32 [lanes], [lanes, depth+1] and [lanes, depth+1]."""
    dev, tokens, ins, outs = _tree_arrays(target_logits, drafts, parents, cu, lanes, depth, V, out_accept_len,
                                          out_commit_ids, out_path)
    _set_stream(dev)
    st = lib.spec_tree_verify(*ins, tokens, lanes, depth, V, *outs)
    if st:
        _check(st)


def spec_tree_verify_sampled(target_logits, drafts, parents, cu, lanes, depth, V, temperature, top_p, top_k, uniforms,
                             out_accept_len, out_commit_ids, out_path):
    """Sampled verify of trees; uniforms float64 [tokens, 2]."""
    dev, tokens, ins, outs = _tree_arrays(target_logits, drafts, parents, cu, lanes, depth, V, out_accept_len,
                                          out_commit_ids, out_path)
    u = _array(uniforms, _torch().float64, 2 * tokens, dev, "uniforms")
    _set_stream(dev)
    st = lib.spec_tree_verify_sampled(*ins, tokens, lanes, depth, V, temperature, top_p, top_k, u, *outs)
    if st:
        _check(st)


def _commit(call, kind, cache, batch, path, accept_lens, depth, context_out):
    _is_cache(cache, kind)
    i32 = _torch().int32
    dev = _on_current_device(cache.device, "cache")
    if batch.device != dev:
        _bad("batch and cache are on different devices")
    p = _array(path, i32, batch.lanes * (_n(depth) + 1), dev, "path")
    a = _array(accept_lens, i32, batch.lanes, dev, "accept_lens")
    c = None if context_out is None else _array(context_out, i32, batch.lanes, dev, "context_out")
    _set_stream(dev)
    st = call(cache._ref, batch._ref, p, a, depth, c)
    if st:
        _check(st)


def spec_tree_commit(cache, batch, path, accept_lens, depth, context_out=None):
    """Move the accepted nodes' keys and values to where a row of tokens has them; the next step's
    context lengths into ``context_out`` int32 [lanes] (or None)."""
    _commit(lib.spec_tree_commit, PagedCache, cache, batch, path, accept_lens, depth, context_out)


def spec_tree_commit8(cache, batch, path, accept_lens, depth, context_out=None):
    """The same in a PagedCache8."""
    _commit(lib.spec_tree_commit8, PagedCache8, cache, batch, path, accept_lens, depth, context_out)


def spec_logits_process(logits, lanes, cols, V, out, *, history=None, prompt_lens=None, history_lens=None,
                        drafts=None, penalties=None, bias_ids=None, bias_vals=None, bias_lens=None, mask=None,
                        mask_rows=None):
    """Penalties, biases and grammar masks on bf16 logits [lanes*cols, V] into
    ``out`` (which may be ``logits``); every rule's tensors may be left out, and
    its tables may have no entries (a history [lanes, 0], say)."""
    t = _torch()
    i32, f32 = t.int32, t.float32
    ln, cs, vs = _n(lanes), _n(cols), _n(V)
    n = ln * cs * vs
    for x, name in ((logits, "logits"), (out, "out")):
        if x is not None and x.dtype is not t.bfloat16 and x.dtype not in (t.int16, t.uint16):
            _bad(f"{name}: dtype {x.dtype} is not bf16 bits")
    dev = t.cuda.current_device()
    lg = None if logits is None else _array(logits, logits.dtype, n, dev, "logits")
    o = None if out is None else _array(out, out.dtype, n, dev, "out")
    if (history is None) != (prompt_lens is None) or (history is None) != (history_lens is None):
        _bad("history, prompt_lens and history_lens go together")
    if (bias_ids is None) != (bias_vals is None) or (bias_ids is None) != (bias_lens is None):
        _bad("bias_ids, bias_vals and bias_lens go together")
    if (mask is None) != (mask_rows is None):
        _bad("mask and mask_rows go together")
    hs = nb = rows = 0
    h = pl = hl = d = pen = bi = bv = bl = m = mr = None
    if history is not None:
        hs = _rows_of(history, ln, "history")
        h = _array(history, i32, ln * hs, dev, "history")
    if prompt_lens is not None:
        pl = _array(prompt_lens, i32, ln, dev, "prompt_lens")
    if history_lens is not None:
        hl = _array(history_lens, i32, ln, dev, "history_lens")
    if drafts is not None:
        d = _array(drafts, i32, ln * (cs - 1), dev, "drafts")
    if penalties is not None:
        pen = _array(penalties, f32, 3 * ln, dev, "penalties")
    if bias_ids is not None:
        nb = _rows_of(bias_ids, ln, "bias_ids")
        bi = _array(bias_ids, i32, ln * nb, dev, "bias_ids")
    if bias_vals is not None:
        bv = _array(bias_vals, f32, ln * nb, dev, "bias_vals")
    if bias_lens is not None:
        bl = _array(bias_lens, i32, ln, dev, "bias_lens")
    if mask is not None:
        words = (vs + 31) // 32
        rows = mask.shape[0]
        if mask.dim() != 2 or mask.shape[1] != words or mask.element_size() != 4:
            _bad(f"mask: need 32-bit words [rows, {words}]")
        m = _array(mask, mask.dtype, rows * words, dev, "mask")
    if mask_rows is not None:
        mr = _array(mask_rows, i32, ln * cs, dev, "mask_rows")
    _set_stream(dev)
    st = lib.spec_logits_process(lg, lanes, cols, V, h, hs, pl, hl, d, pen, bi, bv, nb, bl, m, rows, mr, o)
    if st:
        _check(st)


# ---- allocating conveniences ------------------------------------------------

def paged_attention(q, cache, batch, scale=None, window=0, max_new=0, workspace=None, masks=None):
    """(out, lse) of spec_paged_attention, spec_tree_attention (with ``masks``) or, for a PagedCache8, their 8-bit
    forms; a fresh workspace unless one is given.
    Rows past the step's tokens are not written and hold anything."""
    import torch
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_attention_workspace(q.device)
    scale = cache.head_dim ** -0.5 if scale is None else scale
    eight = isinstance(cache, PagedCache8)
    if masks is None:
        (spec_paged_attention8 if eight else spec_paged_attention)(q, cache, batch, scale, out, lse, workspace, window, max_new)
    else:
        (spec_tree_attention8 if eight else spec_tree_attention)(q, cache, batch, masks, scale, out, lse, workspace, window,
                                                                 max_new)
    return out, lse


def tree_verify(target_logits, drafts, parents, cu, depth, uniforms=None, temperature=1.0, top_p=1.0, top_k=64):
    """(accept_lens, commit_ids, path) of spec_tree_verify or, with uniforms, spec_tree_verify_sampled."""
    import torch
    lanes, V = cu.numel() - 1, target_logits.shape[-1]
    e = lambda *n: torch.empty(n, dtype=torch.int32, device=cu.device)  # noqa: E731
    acc, commit, path = e(lanes), e(lanes, depth + 1), e(lanes, depth + 1)
    if uniforms is None:
        spec_tree_verify(target_logits, drafts, parents, cu, lanes, depth, V, acc, commit, path)
    else:
        spec_tree_verify_sampled(target_logits, drafts, parents, cu, lanes, depth, V, temperature, top_p, min(top_k, V),
                                 uniforms, acc, commit, path)
    return acc, commit, path


def process_logits(logits, lanes, cols, **rules):
    """spec_logits_process into a new tensor of the same shape."""
    import torch
    out = torch.empty_like(logits)
    spec_logits_process(logits, lanes, cols, logits.shape[-1], out, **rules)
    return out
