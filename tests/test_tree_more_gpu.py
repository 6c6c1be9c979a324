"""Calls of the tree and 8-bit cache operators that the main tests do not make: padded steps, other streams, captures
without a call before them, repeated calls, caches past 32 bits of offset.  Needs a GPU."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest

from tests import tree_ref as ref
from tests.test_tree_gpu import _attend, _batch, _cache, _check, _cu, _dt, _i32, _step, _verify_case

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sd():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g
    g._load_build_module().build()
    import speculative_decoding_draft_column_gb300 as sd
    return sd


@pytest.mark.parametrize("eight", [False, True])
def test_rows_past_the_step_are_left(sd, eight):
    """q, masks and out have more rows than the lanes have tokens."""
    import torch
    sizes, ctx, pad, dim, ps = [20, 0, 9], [300, 5, 40], 11, 64, 16
    seq, table, k, v, q = _step(sizes, ctx, 2, 2, dim, ps, "bf16", seed=1)
    cache, (kk, vv) = _cache(sd, k, v, "bf16", eight)
    q = torch.cat([q, torch.full((pad, 4, dim), float("nan"), dtype=q.dtype, device="cuda")])
    cu = _cu(sizes)
    b = _batch(sd, table.tolist(), cu, seq, ps)
    parents = _i32([i // 2 for n in sizes for i in range(n)] + [7] * pad)
    masks = torch.full((len(q), 1), -1, dtype=torch.int32, device="cuda")
    positions = torch.empty(len(q), dtype=torch.int32, device="cuda")
    sd.spec_tree_plan(parents, b, masks, positions)
    assert (masks[cu[-1]:] == 0).all() and (positions[cu[-1]:] == 0).all()
    got, lse = _attend(sd, q, cache, b, masks, 0.125, 0, 20, eight)
    assert (got[cu[-1]:] == 7).all() and (lse[cu[-1]:] == 7).all()
    want = ref.attention(q[:cu[-1]].double().cpu().numpy(), kk, vv, table, cu, seq, masks.cpu().numpy().view(np.uint32), 0.125, 0, "bf16")
    _check(got[:cu[-1]], lse[:cu[-1]], want)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dim,dtype", [(64, "f16"), (128, "bf16"), (256, "bf16")])
def test_equal_calls_give_equal_bits(sd, dim, dtype, tree):
    import torch
    rng = np.random.default_rng(dim)
    sizes = rng.integers(1, 30, 12).tolist()
    ctx = rng.integers(0, 4_000, 12).tolist()
    seq, table, k, v, q = _step(sizes, ctx, 2, 4, dim, 32, dtype, seed=dim)
    cache, _ = _cache(sd, k, v, dtype, True)
    b = _batch(sd, table.tolist(), _cu(sizes), seq, 32)
    masks = torch.tensor(rng.integers(-(1 << 31), 1 << 31, (sum(sizes), 1)), dtype=torch.int32, device="cuda") if tree else None
    first = _attend(sd, q, cache, b, masks, dim ** -0.5, 0, 30, True)
    for _ in range(30):
        again = _attend(sd, q, cache, b, masks, dim ** -0.5, 0, 30, True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_on_another_stream(sd):
    """Inputs made, operators run and results read on a stream that is not the default one."""
    import torch
    rng = np.random.default_rng(3)
    cu, logits, drafts, parents = _verify_case(rng, [12, 7, 30], 9_000, 5)
    want = ref.verify(logits.double().cpu().numpy(), drafts.tolist(), parents, cu, 5)
    seq, table, k, v, q = _step([12, 7, 30], [40, 1_000, 7], 1, 4, 64, 16, "bf16", seed=9)
    cache, _ = _cache(sd, k, v, "bf16", True)
    d, p, c = _i32(drafts.tolist()), _i32(parents), _i32(cu)
    b = _batch(sd, table.tolist(), cu, seq, 16)
    a0, l0 = _attend(sd, q, cache, b, None, 0.125, 0, 30, True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(5_000_000)
        late = logits.clone()
        acc, ids, path = sd.tree_verify(late, d, p, c, 5)
        out, lse = sd.paged_attention(q.clone(), cache, b, scale=0.125, max_new=30)
    s.synchronize()
    assert [x.tolist() for x in (acc, ids, path)] == list(want[:3])
    assert torch.equal(out, a0) and torch.equal(lse, l0)


def test_lanes_that_overlap_leave_the_next_call_alone(sd):
    """cu that decreases says no lanes; nothing is read out of range, and the next call is right."""
    import torch
    rng = np.random.default_rng(6)
    cu, logits, drafts, parents = _verify_case(rng, [5, 4], 6_000, 3)
    want = ref.verify(logits.double().cpu().numpy(), drafts.tolist(), parents, cu, 3)
    d, p = _i32(drafts.tolist()), _i32(parents)
    for bad in ([0, 7, 3, 9], [0, -5, 100, 2], [9, 0, 9, 0]):
        sd.tree_verify(logits, d, p, _i32(bad), 3)
        got = sd.tree_verify(logits, d, p, _i32(cu), 3)
        assert [x.tolist() for x in got] == list(want[:3])
    torch.cuda.synchronize()


@pytest.mark.parametrize("dim,ps", [(128, 64), (256, 16)])
def test_cache_past_32_bits(sd, dim, ps):
    """Pages 2^26 bytes apart: the last ones lie past 2^32."""
    import torch
    pages, heads, n = 70, 2, 40
    big = torch.zeros(pages << 26, dtype=torch.uint8, device="cuda")
    views = [big.as_strided((pages, ps, heads, dim), (1 << 26, heads * dim, dim, 1), at) for at in (0, 1 << 25)]
    scales = [torch.zeros((pages, heads, ps), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = sd.PagedCache8(views[0], scales[0], views[1], scales[1])
    rng = np.random.default_rng(dim)
    need = -(-n // ps)
    table = np.array([[pages - 1 - i for i in range(need)]])
    x = torch.tensor(rng.standard_normal((n, 2 * heads, dim)), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([int(table[0][t // ps]) * ps + t % ps for t in range(n)], device="cuda")
    sd.spec_paged_store8(x[:, :heads], x[:, heads:], slots, cache)
    held = []
    for i in range(2):
        c, e = ref.quantise(x[:, i * heads:(i + 1) * heads].double().cpu().numpy(), "bf16")
        full = np.full((pages, ps, heads, dim), np.nan)
        full[table[0][np.arange(n) // ps], np.arange(n) % ps] = ref.values(c, e)
        held.append(full)
    q = torch.tensor(rng.standard_normal((n, heads * 2, dim)), device="cuda").to(torch.bfloat16)
    b = _batch(sd, table.tolist(), [0, n], [n], ps)
    got, lse = _attend(sd, q, cache, b, None, dim ** -0.5, 0, n, True)
    _check(got, lse, ref.attention(q.double().cpu().numpy(), *held, table, [0, n], [n], None, dim ** -0.5, 0, "bf16"))
    # node 30 to place 1, within pages past 2^32
    before = [views[i][table[0][30 // ps], 30 % ps].clone() for i in range(2)] + [s[table[0][30 // ps], :, 30 % ps].clone() for s in scales]
    sd.spec_tree_commit8(cache, b, _i32([[0, 30]]), _i32([1]), 1)
    after = [views[i][table[0][0], 1] for i in range(2)] + [s[table[0][0], :, 1] for s in scales]
    assert all(torch.equal(x, y) for x, y in zip(before, after))


CAPTURE = """
import torch, sys
sys.path.insert(0, {root!r})
import speculative_decoding_draft_column_gb300 as sd
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
lanes, n, hk, dim, ps, V = 2, 6, 1, 64, 16, 3000
g = torch.Generator("cuda").manual_seed(0)
cache = sd.PagedCache8.create(8, ps, hk, dim)
k, v = (torch.randn((lanes * n, hk, dim), generator=g, device="cuda").bfloat16() for _ in range(2))
q = torch.randn((lanes * n, 2, dim), generator=g, device="cuda").bfloat16()
b = sd.PagedBatch(i32([[0, 1], [2, 3]]), i32([0, n, 2 * n]), i32([n + 9, n]), page_size=ps)
slots = torch.tensor([9 + i if 9 + i < 16 else i - 7 + 16 for i in range(n)] + [32 + i for i in range(n)], device="cuda")
parents = i32([0, 0, 0, 1, 1, 2] * lanes)
logits = (3 * torch.randn((lanes * n, V), generator=g, device="cuda")).bfloat16()
drafts = torch.randint(0, V, (lanes * n,), generator=g, device="cuda", dtype=torch.int32)
drafts[1] = logits[0].float().argmax()
e = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
masks, positions, acc, ids, path, nxt = e(lanes * n, 1), e(lanes * n), e(lanes), e(lanes, 4), e(lanes, 4), e(lanes)
out, lse, ws = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
def step():
    sd.spec_tree_plan(parents, b, masks, positions)
    sd.spec_paged_store8(k, v, slots, cache)
    sd.spec_tree_attention8(q, cache, b, masks, 0.125, out, lse, ws, max_new=n)
    sd.spec_tree_verify(logits, drafts, parents, b.cu_new, lanes, 3, V, acc, ids, path)
    sd.spec_tree_commit8(cache, b, path, acc, 3, nxt)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
cache.k.zero_()
cache.v.zero_()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (masks, positions, out, lse, acc, ids, path, nxt, cache.k, cache.v)]
cache.k.zero_()
cache.v.zero_()
step()
torch.cuda.synchronize()
for x, y in zip(got, (masks, positions, out, lse, acc, ids, path, nxt, cache.k, cache.v)):
    assert torch.equal(x, y)
assert int(acc[0]) >= 1 and sd.spec_device_status() is None
print("as one by one")
"""


def test_first_calls_of_a_process_in_a_capture(sd):
    """Nothing has been called before the capture: no kernel is loaded, no scratch made."""
    r = subprocess.run([sys.executable, "-c", CAPTURE.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as one by one" in r.stdout, r.stderr[-2_000:]
