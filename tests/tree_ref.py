"""Plain float64 forms of the tree and 8-bit cache operators, and the bounds their
results are held to.  Test infrastructure."""
from __future__ import annotations

import math

import numpy as np

from tests.paged_ref import UNIT

NODES = 256


def random_parents(rng, n, deep=1 << 30, chain=False):
    """Parents before children; node 0 the anchor."""
    parents, level = [-1], [0]
    for i in range(1, n):
        p = i - 1 if chain else int(rng.integers(0, i))
        while level[p] >= deep:
            p = parents[p]
        parents.append(p)
        level.append(level[p] + 1)
    return parents


def above(parents):
    """Of each node the set of itself and the nodes above it (a parent that is no earlier node: none)."""
    out = []
    for i, p in enumerate(parents):
        out.append({i} | (out[p] if i and 0 <= p < i else set()))
    return out


def plan(parents, cu, seq, tokens, words):
    """(masks [tokens][words], positions [tokens])"""
    masks, positions = np.zeros((tokens, words), np.uint32), np.zeros(tokens, np.int64)
    for lane in range(len(seq)):
        a, b = cu[lane], cu[lane + 1]
        sets = above([int(p) for p in parents[a:min(b, a + NODES)]])
        for i in range(b - a):
            positions[a + i] = seq[lane] - (b - a)
            if i < NODES:
                positions[a + i] += len(sets[i]) - 1
                for j in sets[i]:
                    if j < 32 * words:
                        masks[a + i, j // 32] |= np.uint32(1 << (j % 32))
    return masks, positions


def seen_keys(masks, ctx, i, window):
    """Keys that node i sees: cached positions (of a window), and the nodes up to i in its mask."""
    nodes = [j for j in range(min(i + 1, 32 * len(masks))) if int(masks[j // 32]) >> (j % 32) & 1]
    lo = max(0, ctx + max(0, len(nodes) - 1) - window + 1) if window else 0
    return list(range(lo, ctx)) + [ctx + j for j in nodes if ctx + j >= 0]


def attention(q, k, v, table, cu, seq, masks, scale, window, dtype):
    """As paged_ref.attention, for rows that see `seen_keys` (masks None: causal).  The bound is the one derived there."""
    T, Hq, D = q.shape
    ps, Hk = k.shape[1], k.shape[2]
    g, u = Hq // Hk, UNIT[dtype]
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    ob, lb = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for lane in range(len(seq)):
        n = cu[lane + 1] - cu[lane]
        ctx = seq[lane] - n
        for i in range(n):
            row = cu[lane] + i
            if masks is None:
                lo = max(0, ctx + i - window + 1) if window else 0
                j = np.arange(lo, ctx + i + 1)
            else:
                j = np.array(seen_keys(masks[row], ctx, i, window), dtype=np.int64)
            if len(j) == 0:
                out[row], lse[row] = 0.0, -np.inf
                continue
            pages = np.asarray(table[lane])[j // ps]
            for h in range(Hk):
                kk, vv = k[pages, j % ps, h], v[pages, j % ps, h]
                for hq in range(h * g, (h + 1) * g):
                    s = scale * (kk @ q[row, hq])
                    m = s.max()
                    w = np.exp(s - m)
                    z = w.sum()
                    w = w / z
                    o = w @ vv
                    A = w @ np.abs(vv)
                    E = 2.0 ** -20 * scale * (np.abs(kk) @ np.abs(q[row, hq])).max()
                    tiny = 2.0 ** -25 * np.abs(vv).sum(0) / z * 256 if dtype == "f16" else 0.0
                    err = (u + 2 * E + 2.0 ** -18) * A + tiny
                    out[row, hq], lse[row, hq] = o, m + np.log(z)
                    ob[row, hq] = u * (np.abs(o) + err) + err + 2.0 ** -25
                    lb[row, hq] = E + 2.0 ** -20 * max(1.0, abs(m + np.log(z)))
    return out, lse, ob, lb


# ---- the 8-bit cache ----------------------------------------------------------

def code_values():
    """What the 256 codes stand for."""
    v = []
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v.append(math.nan if c & 127 == 127 else -x if c & 128 else x)
    return np.array(v)


def least(dtype):
    return -14 if dtype == "f16" else -120


def quantise(x, dtype):
    """(codes, scales) of vectors along the last dimension, float64 of exact 16-bit values."""
    x = np.asarray(x, np.float64)
    codes, scales = np.zeros(x.shape, np.uint8), np.zeros(x.shape[:-1], np.uint8)
    table = code_values()[:127]                       # 0 .. 448, ascending
    for at in np.ndindex(*x.shape[:-1]):
        row = x[at]
        if not np.isfinite(row).all():
            codes[at], scales[at] = 127, 255
            continue
        e = least(dtype)
        while e < 7 and np.abs(row).max() > 448 * 2.0 ** e:
            e += 1
        y = np.minimum(np.abs(row) / 2.0 ** e, 448.0)
        hi = np.searchsorted(table, y).clip(1, 126)
        lo = hi - 1
        dl, dh = y - table[lo], table[hi] - y
        c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        codes[at] = c | np.where(np.signbit(row), 128, 0)
        scales[at] = e + 127
    return codes, scales


def values(codes, scales):
    """What codes [..., n] with scales [...] stand for, float64."""
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return code_values()[codes] * s[..., None]


# ---- verification ---------------------------------------------------------------

def verify(logits, drafts, parents, cu, depth, uniforms=None, temperature=1.0, top_p=1.0, top_k=1):
    """logits float64 [tokens, V].  (accept, commits, path, the smallest distance of a decision from its border)"""
    lanes, margin = len(cu) - 1, math.inf
    accept, commits, paths = [], [], []
    for lane in range(lanes):
        a, n = cu[lane], min(cu[lane + 1] - cu[lane], NODES)
        if n <= 0:
            accept.append(0)
            commits.append([-1] * (depth + 1))
            paths.append([-1] * (depth + 1))
            continue
        cur, ids, path = 0, [], [0]
        while True:
            x = logits[a + cur]
            order = np.lexsort((np.arange(len(x)), -x))[:top_k if uniforms is not None else 1].tolist()
            kids = [i for i in range(1, n) if parents[a + i] == cur] if len(path) <= depth else []
            to = None
            if uniforms is None:
                token = order[0]
                to = next((i for i in kids if drafts[a + i] == token), None)
            else:
                e = [math.exp((x[t] - x[order[0]]) / temperature) for t in order]
                total, run, q = math.fsum(e), 0.0, {}
                for t, y in zip(order, e):
                    q[t] = y / total
                    run += q[t]
                    margin = min(margin, abs(run - top_p))
                    if run >= top_p:
                        break
                whole = math.fsum(q.values())
                q = {t: y / whole for t, y in q.items()}
                for i in kids:
                    t = drafts[a + i]
                    if t not in q:
                        continue
                    goal = uniforms[a + i][0] * math.fsum(q.values())
                    margin = min(margin, abs(goal - q[t]))
                    if goal < q[t]:
                        to, token = i, t
                        break
                    del q[t]
                if to is None:
                    goal, run = uniforms[a + cur][1] * math.fsum(q.values()), 0.0
                    for token, y in q.items():
                        run += y
                        margin = min(margin, abs(run - goal))
                        if run > goal:
                            break
            ids.append(token)
            if to is None:
                break
            path.append(to)
            cur = to
        accept.append(len(path) - 1)
        commits.append(ids + [-1] * (depth + 1 - len(ids)))
        paths.append(path + [-1] * (depth + 1 - len(path)))
    return accept, commits, paths, margin
