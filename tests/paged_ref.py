"""Plain float64 forms of the paged-cache operators and the logits rules, and
the bounds their results are held to.  Test infrastructure."""
from __future__ import annotations

import numpy as np

# unit roundoff of the 16-bit types: bf16 has 8 significant bits, fp16 11
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def plan(ctx, new, held, table, free, cursor, page_size, tokens):
    """Lane by lane, page by page."""
    table = [list(r) for r in table]
    held = list(held)
    most = len(table[0]) if table else 0
    used, short, over, cu, seq = cursor, 0, 0, [0], []
    pos, slots = [], []
    for lane in range(len(ctx)):
        c, n = max(0, ctx[lane]), max(0, new[lane])
        held[lane] = min(max(0, held[lane]), most)
        need = -(-(c + n) // page_size)
        over += need > most
        for _ in range(held[lane], min(need, most)):
            if used < len(free):
                table[lane][held[lane]] = free[used]
                held[lane] += 1
                used += 1
            else:
                short += 1
        for p in range(c, c + n):
            pos.append(p)
            i = p // page_size
            slots.append(table[lane][i] * page_size + p % page_size if i < held[lane] and table[lane][i] >= 0 else -1)
        cu.append(cu[-1] + n)
        seq.append(c + n)
    total = cu[-1]
    pos = (pos + [0] * tokens)[:tokens]
    slots = (slots + [-1] * tokens)[:tokens]
    return table, cu, seq, held, pos, slots, [total, used, short, over]


def attention(q, k, v, table, cu, seq, scale, window, dtype):
    """q [T, Hq, D], k and v [pages, ps, Hk, D], all float64 arrays of exact
    16-bit values.  Returns (out, lse, bound of out, bound of lse); rows no
    lane owns are NaN.

    The bound: the weights round to 16 bits once (u relative, or 2^-25 absolute
    for subnormal fp16 weights against a sum of at least 2^-8 -- a weight is
    taken relative to a maximum that may lag the true one by at most 8 in
    log2), scores carry an fp32 error of E = 2^-20 * max_j sum_i |q_i k_ji| * scale
    (a few times D roundings at 2^-24 of the partial sums), which moves a
    weight and the sum by E relative each, exponentials and fp32 sums are good
    to 2^-18, and the result rounds once."""
    T, Hq, D = q.shape
    ps, Hk = k.shape[1], k.shape[2]
    g, u = Hq // Hk, UNIT[dtype]
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    ob, lb = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for lane in range(len(seq)):
        n = cu[lane + 1] - cu[lane]
        for t in range(n):
            p = seq[lane] - n + t
            row = cu[lane] + t
            lo = max(0, p - window + 1) if window else 0
            if p < lo:
                out[row], lse[row] = 0.0, -np.inf
                continue
            j = np.arange(lo, p + 1)
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


def logits_rules(x, cols, prompt, output, drafts, pen, bias, allowed):
    """One lane: x float64 [cols, V] of exact bf16 values; prompt, output: id
    lists; drafts: ids or None; pen (r, f, p); bias: list of (id, value);
    allowed: per column a boolean array or None."""
    V = x.shape[1]
    x = x.copy()
    r, f, p = pen
    ok = lambda t: 0 <= t < V  # noqa: E731
    asked, count = np.zeros(V, bool), np.zeros(V)
    for t in prompt:
        if ok(t):
            asked[t] = True
    for t in output:
        if ok(t):
            count[t] += 1
    for j in range(cols):
        if j and drafts is not None and ok(drafts[j - 1]):
            count[drafts[j - 1]] += 1
        seen = asked | (count > 0)
        col = x[j]
        col[seen] = np.where(col[seen] > 0, col[seen] / r, col[seen] * r)
        col -= f * count + p * (count > 0)
        for t, b in bias:
            if ok(t):
                col[t] += b
        if allowed[j] is not None:
            col[~allowed[j]] = -np.inf
    return x
