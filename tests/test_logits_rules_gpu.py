"""Penalties, biases and grammar masks on the GPU against the float64 form
(tests/paged_ref.py).  Needs a GPU.

Bound: the rules are at most five fp32 operations (2^-24 relative each, of
terms no larger than |x| * max(r, 1/r) + f * n + p + |bias|), then one
rounding to bf16 (2^-8 of the result)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import paged_ref as ref

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


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _run(sd, lanes, cols, V, hist, seed=0, pen=True, nb=0, mask=False, drafts=True, shift=(0, 0), in_place=False):
    import torch
    rng = np.random.default_rng(seed)
    n = lanes * cols * V
    flat = torch.empty(n + 64, dtype=torch.bfloat16, device="cuda")
    flat[:] = torch.from_numpy(rng.standard_normal(n + 64) * 3).to(torch.bfloat16).cuda()
    guard = torch.full((n + 64,), 5.5, dtype=torch.bfloat16, device="cuda")
    x = flat[8 + shift[0]:8 + shift[0] + n].view(lanes * cols, V)
    y = x if in_place else guard[8 + shift[1]:8 + shift[1] + n].view(lanes * cols, V)
    src = x.double().cpu().numpy().reshape(lanes, cols, V)
    before = flat.clone()
    stride = max(hist, 1)
    whole = rng.integers(0, hist + 1, lanes)
    whole[0] = hist
    prompt = (whole * rng.random(lanes)).astype(int)
    h = (V * rng.random((lanes, stride)) ** 3).astype(int)
    if stride > 3:
        h[:, 0], h[:, 1] = -1, V              # ignored
        h[0, 2:] = V - 1                      # one token many times
    dr = (V * rng.random((lanes, max(cols - 1, 0))) ** 3).astype(int)
    if cols > 2:
        dr[:, 1] = dr[:, 0]                   # a draft repeated
        dr[0, 0] = -1
    p = np.stack([rng.uniform(0.8, 1.5, lanes), rng.uniform(-0.5, 1, lanes), rng.uniform(-0.5, 1, lanes)], 1).astype(np.float32)
    kw = dict(history=_i32(h), prompt_lens=_i32(prompt), history_lens=_i32(whole))
    if pen:
        kw["penalties"] = torch.from_numpy(p).cuda()
    if drafts and cols > 1:
        kw["drafts"] = _i32(dr)
    biases = [[] for _ in range(lanes)]
    if nb:
        ids = np.stack([rng.choice(V, size=nb, replace=V < nb) for _ in range(lanes)])
        vals = rng.standard_normal((lanes, nb)).astype(np.float32) * 4
        if nb > 2:
            vals[:, 0] = -np.inf
            ids[:, 1] = V + 3                 # ignored
        lens = rng.integers(0, nb + 1, lanes)
        lens[0] = nb
        kw.update(bias_ids=_i32(ids), bias_vals=torch.from_numpy(vals).cuda(), bias_lens=_i32(lens))
        biases = [list(zip(ids[l, :lens[l]].tolist(), vals[l, :lens[l]].astype(float).tolist())) for l in range(lanes)]
    allowed = [[None] * cols for _ in range(lanes)]
    if mask:
        words = (V + 31) // 32
        m = rng.integers(0, 1 << 32, (3, words), dtype=np.uint64).astype(np.uint32)
        m[2] = 0                              # a grammar that leaves nothing
        rows = rng.integers(-1, 4, lanes * cols)   # -1 and 3: no mask
        bits = ((m[:, np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1).astype(bool)
        for c in range(lanes * cols):
            if 0 <= rows[c] < 3:
                allowed[c // cols][c % cols] = bits[rows[c]]
        kw.update(mask=torch.from_numpy(m.view(np.int32)).cuda(), mask_rows=_i32(rows))
    sd.spec_logits_process(x, lanes, cols, V, y, **kw)
    torch.cuda.synchronize()
    got = y.double().cpu().numpy().reshape(lanes, cols, V)
    if in_place:
        lo, hi = 8 + shift[0], 8 + shift[0] + n
        assert torch.equal(flat[:lo], before[:lo]) and torch.equal(flat[hi:], before[hi:])
    else:
        lo, hi = 8 + shift[1], 8 + shift[1] + n
        assert (guard[:lo] == 5.5).all() and (guard[hi:] == 5.5).all() and torch.equal(flat, before)
    for l in range(lanes):
        pp = p[l].astype(float) if pen else (1.0, 0.0, 0.0)
        out = h[l, prompt[l]:whole[l]].tolist()
        want = ref.logits_rules(src[l], cols, h[l, :prompt[l]].tolist(), out, dr[l] if "drafts" in kw else None, pp,
                                biases[l], allowed[l])
        inf = np.isinf(want)
        assert np.array_equal(np.where(inf, want, 0.0), np.where(np.isinf(got[l]), got[l], 0.0))
        b = np.zeros(V)
        for t, val in biases[l]:
            if 0 <= t < V and np.isfinite(val):
                b[t] += abs(val)
        size = np.abs(src[l]) * max(pp[0], 1 / pp[0]) + abs(pp[1]) * (len(out) + cols) + abs(pp[2]) + b
        bound = 2.0 ** -8 * np.abs(np.where(inf, 0, want)) + 8 * 2.0 ** -24 * size
        err = np.abs(np.where(inf, 0, got[l]) - np.where(inf, 0, want))
        assert (err <= bound).all(), (l, float((err / bound).max()))


@pytest.mark.parametrize("V", [1, 7, 8, 31, 33, 1_000, 4_088, 4_096, 4_097, 8_191, 12_345])
@pytest.mark.parametrize("cols", [1, 2, 8])
def test_vocabularies(sd, V, cols):
    _run(sd, 3, cols, V, 50, seed=V + cols, nb=min(V, 9), mask=True)
    _run(sd, 1, cols, V, 0, seed=V + cols, mask=True)


@pytest.mark.parametrize("shift", [(0, 0), (1, 1), (3, 3), (7, 7), (0, 1), (5, 2)])
def test_alignments(sd, shift):
    _run(sd, 2, 3, 5_003, 100, seed=sum(shift), nb=5, mask=True, shift=shift)
    _run(sd, 2, 3, 5_003, 100, seed=sum(shift), nb=5, mask=True, shift=shift, in_place=True)


def test_each_rule_alone(sd):
    for kw in (dict(pen=True), dict(pen=False, nb=40), dict(pen=False, mask=True), dict(pen=True, drafts=False),
               dict(pen=False)):
        _run(sd, 2, 4, 9_001, 300, seed=11, **kw)


def test_repeated_biases_add_up_in_order(sd):
    """Sums whose value depends on the order: those of fp32 additions from the first to the last, in every call."""
    import torch
    V, nb = 9_000, 700
    rng = np.random.default_rng(5)
    ids = rng.choice([3, 17, 4_095, 4_096, 8_999], size=(2, nb)).astype(np.int32)
    ids[1, :3] = -1, V, 5_000                 # two of no token, one given once
    vals = (rng.standard_normal((2, nb)) * 10.0 ** rng.integers(-3, 8, (2, nb))).astype(np.float32)
    lens = [nb, nb - 1]
    want = np.zeros((2, V), dtype=np.float32)
    for l in range(2):
        for t, v in zip(ids[l, :lens[l]], vals[l, :lens[l]]):
            if 0 <= t < V:
                want[l, t] = np.float32(want[l, t] + v)
    x = torch.zeros((2, V), dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        y = sd.process_logits(x, 2, 1, bias_ids=_i32(ids), bias_vals=torch.from_numpy(vals).cuda(), bias_lens=_i32(lens))
        assert torch.equal(y, torch.from_numpy(want).to(torch.bfloat16).cuda())


def test_largest_block(sd):
    _run(sd, 5, 16, 20_011, 5_000, seed=3, nb=300, mask=True)


def test_full_vocabulary_feeds_verify(sd):
    """A mask that leaves one token makes the verify commit it."""
    import torch
    lanes, gamma, V = 2, 3, sd.SPEC_VOCAB
    x = torch.randn((lanes * (gamma + 1), V), device="cuda").to(torch.bfloat16)
    words = (V + 31) // 32
    only = [17, 200_000, 248_045, 31, 32, 99_999, 5, 131_072]
    m = np.zeros((8, words), dtype=np.uint32)
    for c, t in enumerate(only):
        m[c, t // 32] = np.uint32(1 << (t % 32))
    y = sd.process_logits(x, lanes, gamma + 1, mask=torch.from_numpy(m.view(np.int32)).cuda(), mask_rows=_i32(range(8)))
    drafts = _i32([only[0:3], [only[4], 1, 1]]).view(2, 3)
    acc, com = sd.verify(y, drafts)
    assert acc.cpu().tolist() == [3, 1]
    assert com.cpu().tolist() == [only[:4], only[4:6] + [-1, -1]]


def test_no_lanes(sd):
    import torch
    e = torch.empty((0, 10), dtype=torch.bfloat16, device="cuda")
    sd.spec_logits_process(e, 0, 1, 10, e)
