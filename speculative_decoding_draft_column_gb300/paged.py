"""Binding of the paged cache and the logits rules (see ``include/specsel.h``).

``PagedCache`` and ``PagedBatch`` describe a caller's tensors to the library:
they check them once, keep them alive and hold the C struct; they own no data
of their own unless made with ``create``.  The calls check what changes from
call to call, set the library's stream to PyTorch's current one and forward to
the C entry point of the same name.
"""
from __future__ import annotations

import ctypes

from . import SPEC_ERR_ARG, SpecError, _check, _dev, _n, _use_torch_stream, lib

SPEC_BF16, SPEC_F16 = 0, 1
SPEC_PAGED_MAX_LANES = 4096

_p, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_strides", _i64 * 3), ("v_strides", _i64 * 3), ("pages", _i64),
                ("page_size", _i32), ("heads", _i32), ("head_dim", _i32), ("dtype", _i32)]


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


def _typed(x, dtype, count, name):
    """Pointer of a contiguous CUDA tensor of `dtype` with at least `count` elements."""
    if x.dtype != dtype:
        _bad(f"{name}: dtype {x.dtype}, need {dtype}")
    return _dev(x, count, x.element_size(), name)


def _strided(x, shape, cache, name):
    """Check a [tokens, heads, head_dim] tensor whose rows are contiguous."""
    if not x.is_cuda or x.device.index != cache.device:
        _bad(f"{name}: on {x.device}, the cache is on cuda:{cache.device}")
    if x.dtype != cache.torch_dtype:
        _bad(f"{name}: dtype {x.dtype}, the cache's is {cache.torch_dtype}")
    if x.dim() != 3 or (shape is not None and tuple(x.shape) != shape) or x.shape[2] != cache.head_dim:
        _bad(f"{name}: shape {tuple(x.shape)}, need {shape or ('tokens', 'heads', cache.head_dim)}")
    if x.stride(2) != 1 and x.numel():
        _bad(f"{name}: the last dimension must be contiguous")


def _on_current_device(index, name):
    import torch
    if index != torch.cuda.current_device():
        _bad(f"{name}: on cuda:{index}, the current device is cuda:{torch.cuda.current_device()}")


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
        i32 = torch.int32
        s = _BatchStruct(block_table=_typed(block_table, i32, lanes * max_pages, "block_table"),
                         cu_new=_typed(cu_new, i32, lanes + 1, "cu_new"),
                         seq_lens=_typed(seq_lens, i32, lanes, "seq_lens"),
                         lanes=lanes, max_pages=max_pages, page_size=page_size)
        self.device = block_table.device.index
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
                setattr(s, name, _typed(getattr(self, name), i32, count, name))
            s.slots = _typed(slots, torch.int64, tokens, "slots")
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
    int32 [1] (the pages of the list used before) or None."""
    import torch
    if not batch.plannable:
        _bad("batch: made without the plan's buffers")
    _on_current_device(batch.device, "batch")
    n = free_pages.numel()
    f = _typed(free_pages, torch.int32, n, "free_pages")
    c = None if cursor is None else _typed(cursor, torch.int32, 1, "cursor")
    _use_torch_stream()
    _check(lib.spec_paged_plan(batch._ref, f, n, c))


def spec_paged_store(k, v, slots, cache):
    """Store k, v [tokens, heads, head_dim] at slots int64 [tokens] of the cache."""
    import torch
    tokens = k.shape[0]
    shape = (tokens, cache.heads, cache.head_dim)
    _strided(k, shape, cache, "k")
    _strided(v, shape, cache, "v")
    _on_current_device(cache.device, "cache")
    sl = _typed(slots, torch.int64, tokens, "slots")
    _use_torch_stream()
    _check(lib.spec_paged_store(k.data_ptr(), v.data_ptr(), tokens, k.stride(0), k.stride(1), v.stride(0),
                                v.stride(1), sl, cache._ref))


def spec_paged_attention_workspace() -> int:
    """Bytes of workspace an attention call needs on the current device."""
    n = int(lib.spec_paged_attention_workspace())
    if n < 0:
        _check(n)
    return n


def new_attention_workspace(device="cuda"):
    """A zeroed workspace for spec_paged_attention (one per stream that may run it)."""
    import torch
    with torch.cuda.device(device):
        return torch.zeros(spec_paged_attention_workspace(), dtype=torch.uint8, device=device)


def spec_paged_attention(q, cache, batch, scale, out, lse, workspace, window=0, max_new=0):
    """Attention of the batch's new tokens: q [tokens, heads_q, head_dim] into
    out (same shape, contiguous) and lse fp32 [tokens, heads_q] (or None)."""
    import torch
    _strided(q, None, cache, "q")
    _on_current_device(cache.device, "cache")
    if batch.device != cache.device:
        _bad("batch and cache are on different devices")
    tokens, heads_q, _ = q.shape
    if out.dtype != cache.torch_dtype or out.shape != q.shape:
        _bad(f"out: {out.dtype} {tuple(out.shape)}, need {cache.torch_dtype} {tuple(q.shape)}")
    o = _dev(out, q.numel(), 2, "out")
    ls = None if lse is None else _typed(lse, torch.float32, tokens * heads_q, "lse")
    ws = _dev(workspace, 0, 1, "workspace")
    _use_torch_stream()
    _check(lib.spec_paged_attention(q.data_ptr(), tokens, heads_q, q.stride(0), q.stride(1), cache._ref, batch._ref,
                                    scale, window, max_new, o, ls, ws,
                                    workspace.numel() * workspace.element_size()))


def spec_logits_process(logits, lanes, cols, V, out, *, history=None, prompt_lens=None, history_lens=None,
                        drafts=None, penalties=None, bias_ids=None, bias_vals=None, bias_lens=None, mask=None,
                        mask_rows=None):
    """Penalties, biases and grammar masks on bf16 logits [lanes*cols, V] into
    ``out`` (which may be ``logits``); every rule's tensors may be left out."""
    import torch
    i32 = torch.int32
    ln, cs, n = _n(lanes), _n(cols), _n(lanes) * _n(cols) * _n(V)
    for x, name in ((logits, "logits"), (out, "out")):
        if x is not None and x.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
            _bad(f"{name}: dtype {x.dtype} is not bf16 bits")
    lg, o = _dev(logits, n, 2, "logits"), _dev(out, n, 2, "out")
    hs = nb = rows = 0
    h = pl = hl = d = pen = bi = bv = bl = m = mr = None
    if history is not None:
        if history.dim() != 2 or history.shape[0] < ln:
            _bad("history: need [lanes, length]")
        hs = history.shape[1]
        h = _typed(history, i32, ln * hs, "history")
    if prompt_lens is not None:
        pl = _typed(prompt_lens, i32, ln, "prompt_lens")
    if history_lens is not None:
        hl = _typed(history_lens, i32, ln, "history_lens")
    if drafts is not None:
        d = _typed(drafts, i32, ln * (cs - 1), "drafts")
    if penalties is not None:
        pen = _typed(penalties, torch.float32, 3 * ln, "penalties")
    if bias_ids is not None:
        if bias_ids.dim() != 2 or bias_ids.shape[0] < ln:
            _bad("bias_ids: need [lanes, biases]")
        nb = bias_ids.shape[1]
        bi = _typed(bias_ids, i32, ln * nb, "bias_ids")
    if bias_vals is not None:
        bv = _typed(bias_vals, torch.float32, ln * nb, "bias_vals")
    if bias_lens is not None:
        bl = _typed(bias_lens, i32, ln, "bias_lens")
    if mask is not None:
        words = (_n(V) + 31) // 32
        if mask.dim() != 2 or mask.shape[1] != words or mask.element_size() != 4:
            _bad(f"mask: need 32-bit words [rows, {words}]")
        rows = mask.shape[0]
        m = _dev(mask, rows * words, 4, "mask")
    if mask_rows is not None:
        mr = _typed(mask_rows, i32, ln * cs, "mask_rows")
    _use_torch_stream()
    _check(lib.spec_logits_process(lg, lanes, cols, V, h, hs, pl, hl, d, pen, bi, bv, nb, bl, m, rows, mr, o))


# ---- allocating conveniences ------------------------------------------------

def paged_attention(q, cache, batch, scale=None, window=0, max_new=0, workspace=None):
    """(out, lse) of spec_paged_attention; a fresh workspace unless one is given."""
    import torch
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_attention_workspace(q.device)
    spec_paged_attention(q, cache, batch, cache.head_dim ** -0.5 if scale is None else scale, out, lse, workspace,
                         window, max_new)
    return out, lse


def process_logits(logits, lanes, cols, **rules):
    """spec_logits_process into a new tensor of the same shape."""
    import torch
    out = torch.empty_like(logits)
    spec_logits_process(logits, lanes, cols, logits.shape[-1], out, **rules)
    return out
