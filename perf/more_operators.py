"""Cases of the operators for rounds whose drafts form a tree, and of the 8-bit
paged cache: attention of a tree of drafts over the cache, verification of the
tree against the target, the accepted path moved into place, new keys and
values quantised as they are stored, and attention that reads them back.

A lane's step is a tree of nodes: node 0 is the anchor (the lane's last
committed token), every other node a draft that follows its parent.  The lanes'
nodes lie one after the other, parents before their children.  Trees and
lengths follow from the case alone (its "pick"), values from the seed.
"""
import math
import random

import torch

own = False

VOCAB = 248_046          # the target's output head
SHORTLIST = 131_072      # the shortlist head
WINDOW = 2_048           # the drafter's sliding window
TEMPERATURE, TOP_P, TOP_K = 1.0, 0.95, 20

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one lane, an anchor and fifteen drafts after a short prompt: the smallest tree step, where latency counts
        attention("tree 1x16", 1, 16, 16, 5, 1_013, 1_013, 32, 8, 128, 16, "bf16", 0, False, 1),
        # eight lanes of full trees over mixed contexts, on the 8-bit cache
        attention("tree 8x64 on 8 bits", 8, 64, 64, 8, 500, 16_000, 32, 8, 128, 64, "bf16", 0, True, 2),
        # a drafter's layer over ragged trees: small heads, half precision, a sliding window
        attention("tree drafter 32 lanes", 32, 4, 48, 6, 100, 6_000, 16, 2, 64, 32, "f16", WINDOW, False, 3),
        # many lanes decoding one token each from the 8-bit cache
        attention("decode 64x1 on 8 bits", 64, 1, 1, 0, 500, 16_000, 32, 8, 128, 64, "bf16", 0, True, 4),
        # one lane verifying an anchor and fifteen drafts in a row at the longest context, on the 8-bit cache
        attention("verify 1x16 on 8 bits", 1, 16, 16, 0, 262_128, 262_128, 32, 8, 128, 128, "bf16", 0, True, 5),
        # the new keys and values of a small verify step, quantised
        store("store 8x8", 64, 8, 128, 64, 8, "bf16", 1),
        # those of a large batch of prompt chunks, some tokens without a page
        store("store 16384", 16_384, 8, 128, 64, 512, "bf16", 2),
        # one lane, greedy: the smallest tree to verify
        verify("greedy 1x16", 1, 16, 16, 5, VOCAB, False, 1),
        # eight lanes of full trees, sampled
        verify("sampled 8x64", 8, 64, 64, 8, VOCAB, True, 2),
        # a large batch of ragged trees, sampled
        verify("sampled 64 ragged", 64, 8, 32, 6, VOCAB, True, 3),
        # the accepted paths of a small round moved into place
        commit("commit 8x64", 8, 64, 64, 8, 100, 1_000, 8, 128, 64, "bf16", False, 1),
        # those of a large batch, on the 8-bit cache
        commit("commit 256 on 8 bits", 256, 8, 32, 6, 50, 400, 8, 128, 64, "bf16", True, 2),
    ]


def attention(name, lanes, nodes_lo, nodes_hi, depth, ctx_lo, ctx_hi, heads_q, heads_kv, dim, page, dtype, window,
              eight, pick):
    """Attention of each lane's new tokens over its cached ones and themselves: a tree `depth` deep at most, or
    tokens in a row (depth 0); `eight`: the cache in 8 bits."""
    return {"name": name, "op": "attention", "lanes": lanes, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi,
            "depth": depth, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "heads_q": heads_q, "heads_kv": heads_kv, "dim": dim,
            "page": page, "dtype": dtype, "window": window, "eight": eight, "pick": pick}


def store(name, tokens, heads_kv, dim, page, pages, dtype, pick):
    """New keys and values into their slots of an 8-bit paged cache."""
    return {"name": name, "op": "store", "tokens": tokens, "heads_kv": heads_kv, "dim": dim, "page": page,
            "pages": pages, "dtype": dtype, "pick": pick}


def verify(name, lanes, nodes_lo, nodes_hi, depth, vocab, sampled, pick):
    """Trees of drafts against the target's logits of every node: greedy, or sampled with given uniforms."""
    return {"name": name, "op": "verify", "lanes": lanes, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "depth": depth,
            "vocab": vocab, "sampled": sampled, "pick": pick}


def commit(name, lanes, nodes_lo, nodes_hi, depth, ctx_lo, ctx_hi, heads_kv, dim, page, dtype, eight, pick):
    """Keys and values of the accepted nodes moved to where a row of tokens has them."""
    return {"name": name, "op": "commit", "lanes": lanes, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "depth": depth,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "heads_kv": heads_kv, "dim": dim, "page": page, "dtype": dtype,
            "eight": eight, "pick": pick}


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    pick = rng.randrange(1 << 30)
    op = rng.choice(["attention", "attention", "attention", "verify", "verify", "store", "commit"])
    heads_kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    page, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "bf16", "f16"])
    lanes, nodes_hi, depth = _log(rng, 1, 64), _log(rng, 2, 64), rng.randint(1, 12)
    nodes_lo = rng.choice([1, max(1, nodes_hi // 2), nodes_hi])
    if op == "attention":
        group = rng.choice([1, 2, 3, 4, 5, 8])
        window = rng.choice([0, 0, 0, WINDOW, _log(rng, 256, 8_192)])
        eight = rng.random() < 0.6
        if eight and rng.random() < 0.5:       # tokens in a row: decoding, drafts of a chain, pieces of a prompt
            depth = 0
            nodes_lo = nodes_hi = rng.choice([1, 8, _log(rng, 2, 2_048)])
            lanes = min(lanes, max(1, 4_096 // nodes_hi))
        most = min(262_128, 8_000_000 // (lanes * heads_kv), 1_000_000_000 // (lanes * nodes_hi * heads_kv * group))
        ctx_hi = _log(rng, 40, max(64, most))
        return attention("", lanes, nodes_lo, nodes_hi, depth, rng.choice([0, ctx_hi // 4, ctx_hi]), ctx_hi,
                         heads_kv * group, heads_kv, dim, page, dtype, window, eight, pick)
    if op == "verify":
        vocab = rng.choice([VOCAB, VOCAB, SHORTLIST, _log(rng, 1_001, 248_045)])
        return verify("", lanes, nodes_lo, min(nodes_hi, 2_048 // lanes), depth, vocab, rng.random() < 0.6, pick)
    if op == "store":
        tokens = _log(rng, 1, 16_384 * 8 * 128 // max(8 * 128, heads_kv * dim))
        return store("", tokens, heads_kv, dim, page, -(-tokens * 2 // page) + 1, dtype, pick)
    return commit("", _log(rng, 1, 256), nodes_lo, nodes_hi, depth, 0, _log(rng, 10, 400), heads_kv, dim, page, dtype,
                  rng.random() < 0.5, pick)


# ---- lengths and trees: from the case alone ---------------------------------

def _trees(case):
    """(parents of each lane's nodes, the path that the target agrees with, cached tokens) of each lane."""
    rng = random.Random(case["pick"])
    lo, hi = min(case["nodes_lo"], case["nodes_hi"]), case["nodes_hi"]
    sizes = [rng.randint(lo, hi) for _ in range(case["lanes"])]
    sizes[rng.randrange(len(sizes))] = hi
    ctx = [rng.randint(case.get("ctx_lo", 0), case.get("ctx_hi", 0)) for _ in range(case["lanes"])]
    ctx[rng.randrange(len(ctx))] = case.get("ctx_hi", 0)
    lanes = []
    for n, c in zip(sizes, ctx):
        parents, level = [-1], [0]
        for i in range(1, n):
            p = i - 1
            if case["depth"]:
                # drafts are likelier below the first ones of a level
                p = min(rng.randrange(i), rng.randrange(i))
                while level[p] >= case["depth"]:
                    p = parents[p]
            parents.append(p)
            level.append(level[p] + 1)
        path = [0]
        while rng.random() < 0.75:             # how often one of a node's drafts is right
            below = [i for i in range(path[-1] + 1, n) if parents[i] == path[-1]]
            if not below:
                break
            path.append(below[0] if rng.random() < 0.6 else rng.choice(below))
        lanes.append((parents, path, c))
    return lanes


def _levels(parents):
    level = [0]
    for p in parents[1:]:
        level.append(level[p] + 1)
    return level


def _columns(case):
    """Nodes in the widest row of a mask, in 32-bit words."""
    return -(-case["nodes_hi"] // 32)


def work(case):
    lanes = _trees(case) if case["op"] != "store" else []
    if case["op"] == "attention":
        w, g = case["window"] or 1 << 62, case["heads_q"] // case["heads_kv"]
        keys = pairs = pages = 0
        for parents, _, c in lanes:
            n = len(parents)
            first = max(0, c - w + 1)
            keys += c + n - first
            pairs += sum(min(c + d + 1, w) for d in _levels(parents))
            pages += -(-(c + n) // case["page"]) - first // case["page"]
        rows = sum(len(p) for p, _, _ in lanes)
        vector = case["dim"] + 1 if case["eight"] else 2 * case["dim"]
        moved = keys * case["heads_kv"] * vector * 2 + rows * case["heads_q"] * (case["dim"] * 4 + 4) + 4 * pages \
            + 8 * case["lanes"]
        if case["depth"]:
            moved += rows * (4 + 4 + 4 * _columns(case))
        return {"bytes": moved, "flops": 4 * pairs * case["heads_kv"] * g * case["dim"]}
    if case["op"] == "verify":
        # a column for every node of the path, the drafts' tokens and parents, commits and paths
        columns, nodes = sum(len(path) for _, path, _ in lanes), sum(len(p) for p, _, _ in lanes)
        return {"bytes": columns * case["vocab"] * 2 + 8 * nodes + case["lanes"] * (8 + 8 * (case["depth"] + 1)),
                "flops": columns * case["vocab"]}
    if case["op"] == "commit":
        moves = sum(sum(i != at for i, at in enumerate(path)) for _, path, _ in lanes)
        vector = case["dim"] + 1 if case["eight"] else 2 * case["dim"]
        return {"bytes": moves * case["heads_kv"] * vector * 4 + 8 * moves
                + case["lanes"] * (16 + 4 * (case["depth"] + 1)), "flops": 0}
    kept = case["tokens"] - case["tokens"] // 16
    return {"bytes": kept * case["heads_kv"] * (case["dim"] * 6 + 2) + 8 * case["tokens"],
            "flops": 4 * kept * case["heads_kv"] * case["dim"]}


# ---- inputs -----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + case["pick"] % 999_983)
    s = {"case": case}
    if case["op"] != "store":
        _prepare_lanes(case, s)
    {"attention": _prepare_attention, "verify": _prepare_verify, "commit": _prepare_commit,
     "store": _prepare_store}[case["op"]](case, g, s)
    if own:   # the handles that a program makes once, of its own buffers: pointers and sizes, no data
        _handles(case, s)
    return s


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _least(dtype):
    """The smallest exponent of a vector's scale: what the 16-bit type can multiply by without loss."""
    return -14 if dtype is torch.float16 else -120


def _quantise(x):
    """Codes (e4m3) and exponents of vectors along the last dimension: the smallest power of two that brings the
    vector's largest value to 448 or below; values round to the nearest code, ties to even."""
    largest = x.float().abs().amax(-1)
    m, e = torch.frexp(largest)
    e = torch.where(largest > 0, e - 9 + (m > 0.875).int(), _least(x.dtype)).clamp(_least(x.dtype), 7)
    scaled = torch.ldexp(x.float(), -e[..., None])
    return scaled.clamp(-448, 448).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _new_cache(case, g, s, pages):
    """Keys and values of `pages` pages: 16-bit, or 8-bit codes with a byte of scale a vector."""
    shape = (pages, case["page"], case["heads_kv"], case["dim"])
    s["caches"] = []
    for _ in range(2):
        x = _normal(g, shape, _DTYPES[case["dtype"]])
        if not case.get("eight", True):
            s["caches"].append(x)
            continue
        codes, scales = _quantise(x)
        s["caches"] += [codes, scales.transpose(1, 2).contiguous()]


def _prepare_lanes(case, s):
    lanes = _trees(case)
    cu = [0]
    for parents, _, _ in lanes:
        cu.append(cu[-1] + len(parents))
    s["nodes"] = [len(p) for p, _, _ in lanes]
    s["parents"] = _int32([p for parents, _, _ in lanes for p in parents])
    s["cu_new"], s["new_lens"] = _int32(cu), _int32(s["nodes"])
    s["seq_lens"] = _int32([c + len(p) for p, _, c in lanes])
    s["tokens"] = cu[-1]


def _prepare_table(case, g, s):
    p = case["page"]
    need = [-(-(c + len(t)) // p) for t, _, c in _trees(case)]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((case["lanes"], max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for lane, n in enumerate(need):
        table[lane, :n] = perm[at:at + n]
        at += n
    s["block_table"] = table
    _new_cache(case, g, s, pages)


def _prepare_attention(case, g, s):
    _prepare_table(case, g, s)
    s["q"] = _normal(g, (s["tokens"], case["heads_q"], case["dim"]), _DTYPES[case["dtype"]])
    s["scale"] = case["dim"] ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((s["tokens"], case["heads_q"]), dtype=torch.float32, device="cuda")
    if case["depth"]:
        s["masks"] = torch.empty((s["tokens"], _columns(case)), dtype=torch.int32, device="cuda")
        s["positions"] = torch.empty(s["tokens"], dtype=torch.int32, device="cuda")


def _prepare_verify(case, g, s):
    v = case["vocab"]
    s["logits"] = (3 * _normal(g, (s["tokens"], v), torch.float32)).to(torch.bfloat16)
    s["drafts"] = torch.randint(0, v, (s["tokens"],), generator=g, device="cuda", dtype=torch.int32)
    # the target agrees with each path: its next token stands out of the column before it
    first, row, node = 0, [], []
    for parents, path, _ in _trees(case):
        row += [first + i for i in path[:-1]]
        node += [first + i for i in path[1:]]
        first += len(parents)
    if row:
        row, node = (torch.tensor(x, device="cuda") for x in (row, node))
        s["logits"][row, s["drafts"][node].long()] = 17 + _normal(g, (row.numel(),), torch.float32).to(torch.bfloat16)
    s["uniforms"] = torch.rand((s["tokens"], 2), generator=g, device="cuda", dtype=torch.float64)
    lanes, width = case["lanes"], case["depth"] + 1
    e32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    s["accept"], s["ids"], s["path"] = e32(lanes), e32(lanes, width), e32(lanes, width)


def _prepare_commit(case, g, s):
    _prepare_table(case, g, s)
    width = case["depth"] + 1
    paths = [path[:width] for _, path, _ in _trees(case)]
    s["path"] = _int32([p + [-1] * (width - len(p)) for p in paths])
    s["accept"] = _int32([len(p) - 1 for p in paths])
    s["context"] = torch.empty(case["lanes"], dtype=torch.int32, device="cuda")


def _prepare_store(case, g, s):
    _new_cache(case, g, s, case["pages"])
    # a layer's projections give queries, keys and values side by side: keys and values are strided views; heads
    # differ in size
    t, h, d = case["tokens"], case["heads_kv"], case["dim"]
    size = torch.exp2(torch.randint(-6, 7, (t, 2 * h, 1), generator=g, device="cuda").float())
    kv = (_normal(g, (t, 2 * h, d), torch.float32) * size).to(_DTYPES[case["dtype"]])
    s["k"], s["v"] = kv[:, :h], kv[:, h:]
    slots = torch.randperm(case["pages"] * case["page"], generator=g, device="cuda")[:t]
    gone = torch.randperm(t, generator=g, device="cuda")[:t // 16]
    slots[gone] = -1
    s["slots"] = slots.to(torch.int64).contiguous()


# ---- the framework's operators ----------------------------------------------

def _handles(case, s):
    import speculative_decoding_draft_column_gb300 as sd
    if "caches" in s:
        c = s["caches"]
        s["cache"] = sd.PagedCache8(*c, dtype=_DTYPES[case["dtype"]]) if len(c) == 4 else sd.PagedCache(*c)
    if "block_table" in s:
        s["batch"] = sd.PagedBatch(s["block_table"], s["cu_new"], s["seq_lens"], page_size=case["page"])
    if case["op"] == "attention":
        s["workspace"] = sd.new_attention_workspace()


def run(state):
    op = state["case"]["op"]
    return {"attention": _run_attention, "verify": _run_verify, "commit": _run_commit, "store": _run_store}[op](state)


def _run_attention(s):
    c = s["case"]
    if own:
        import speculative_decoding_draft_column_gb300 as sd
        if c["depth"]:
            sd.spec_tree_plan(s["parents"], s["batch"], s["masks"], s["positions"])
            tree = sd.spec_tree_attention8 if c["eight"] else sd.spec_tree_attention
            tree(s["q"], s["cache"], s["batch"], s["masks"], s["scale"], s["out"], s["lse"], s["workspace"],
                 window=c["window"], max_new=c["nodes_hi"])
            return s["out"], s["lse"], s["masks"], s["positions"]
        sd.spec_paged_attention8(s["q"], s["cache"], s["batch"], s["scale"], s["out"], s["lse"], s["workspace"],
                                 window=c["window"], max_new=c["nodes_hi"])
        return s["out"], s["lse"]
    return _plain_attention(s)


def _run_verify(s):
    c = s["case"]
    if own:
        import speculative_decoding_draft_column_gb300 as sd
        if c["sampled"]:
            sd.spec_tree_verify_sampled(s["logits"], s["drafts"], s["parents"], s["cu_new"], c["lanes"], c["depth"],
                                        c["vocab"], TEMPERATURE, TOP_P, TOP_K, s["uniforms"], s["accept"], s["ids"],
                                        s["path"])
        else:
            sd.spec_tree_verify(s["logits"], s["drafts"], s["parents"], s["cu_new"], c["lanes"], c["depth"],
                                c["vocab"], s["accept"], s["ids"], s["path"])
        return s["accept"], s["ids"], s["path"]
    return _plain_verify(s)


def _run_commit(s):
    c = s["case"]
    if own:
        import speculative_decoding_draft_column_gb300 as sd
        move = sd.spec_tree_commit8 if c["eight"] else sd.spec_tree_commit
        move(s["cache"], s["batch"], s["path"], s["accept"], c["depth"], s["context"])
        return s["caches"], s["context"]
    return _plain_commit(s)


def _run_store(s):
    if own:
        import speculative_decoding_draft_column_gb300 as sd
        sd.spec_paged_store8(s["k"], s["v"], s["slots"], s["cache"])
        return s["caches"]
    return _plain_store(s)


# ---- plain forms ------------------------------------------------------------

def _padded(s):
    """Rows [lanes, most] of the lanes' nodes in the flat arrays, and which of them are there."""
    t = torch.arange(max(s["nodes"]), device=s["cu_new"].device)
    at = s["cu_new"][:-1, None].long() + t
    return at.clamp(max=s["tokens"] - 1), t < s["new_lens"][:, None]


def _ancestors(s, rows, there):
    """[lanes, n, n]: whether node j is node i or above it, by squaring the step to the parent."""
    n = rows.shape[1]
    parents = torch.where(there, s["parents"][rows].long(), -1)
    parents[:, 0] = -1
    eye = torch.eye(n, device=rows.device)
    up = (parents[..., None] == torch.arange(n, device=rows.device)).float() + eye
    for _ in range(max(1, (n - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    return up > 0


def _read(s, pages):
    """Keys and values of pages [lanes, m] in 32 bits: two of [lanes, keys, heads, dim]."""
    c = s["case"]
    if c["eight"]:
        codes, scales = s["caches"][0::2], s["caches"][1::2]
        # (the codes as bytes: the library indexes no 8-bit floats)
        both = [torch.ldexp(k.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float(),
                            e[pages].int().transpose(-1, -2)[..., None] - 127) for k, e in zip(codes, scales)]
    else:
        both = [x[pages].float() for x in s["caches"]]
    return [x.view(pages.shape[0], -1, c["heads_kv"], c["dim"]) for x in both]


def _plain_attention(s):
    """All lanes at once, padded to the largest tree and the longest context."""
    c = s["case"]
    lanes, hk, d = c["lanes"], c["heads_kv"], c["dim"]
    g = c["heads_q"] // hk
    rows, there = _padded(s)
    n, dev = rows.shape[1], rows.device
    q = s["q"][rows].float().view(lanes, n, hk, g, d).permute(0, 2, 3, 1, 4)
    k, v = _read(s, s["block_table"].long())
    keys = k.shape[1]
    x = torch.matmul(q.reshape(lanes, hk, g * n, d), k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(lanes, hk, g, n, keys)
    ctx = (s["seq_lens"] - s["new_lens"]).long()
    j = torch.arange(keys, device=dev)
    if c["depth"]:
        up = _ancestors(s, rows, there)
        deep = up.sum(-1) - 1
        node = j - ctx[:, None]                                            # [lanes, keys]
        seen = torch.gather(up, 2, node.clamp(0, n - 1)[:, None].expand(lanes, n, keys))
        hidden = (node >= 0)[:, None] & ~(seen & (node < n)[:, None])
    else:
        deep = torch.arange(n, device=dev).expand(lanes, n)
        hidden = j > (ctx[:, None] + deep)[..., None]
    if c["window"]:
        hidden |= (j <= (ctx[:, None] + deep - c["window"])[..., None]) & (j < ctx[:, None, None] if c["depth"] else True)
    x.masked_fill_(hidden[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(lanes, hk, g * n, keys), v.permute(0, 2, 1, 3)).view(lanes, hk, g, n, d) / z
    lse = (m + z.log()).squeeze(-1)
    out, total = s["out"], s["lse"]
    out[rows[there]] = o.permute(0, 3, 1, 2, 4).reshape(lanes, n, hk * g, d)[there].to(out.dtype)
    total[rows[there]] = lse.permute(0, 3, 1, 2).reshape(lanes, n, hk * g)[there]
    if not c["depth"]:
        return out, total
    words = _columns(c)
    bits = torch.zeros((lanes, n, 32 * words), dtype=torch.int64, device=dev)
    bits[..., :n] = up
    w = (bits.view(lanes, n, words, 32) << torch.arange(32, device=dev)).sum(-1)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w)[there].int()
    return out, total, w, (ctx[:, None] + deep)[there].int()


def _plain_verify(s):
    """A level of all lanes at a time, decisions in 64 bits (a uniform may lie next to a border)."""
    c = s["case"]
    lanes, v, depth = c["lanes"], c["vocab"], c["depth"]
    rows, there = _padded(s)
    n, dev = rows.shape[1], rows.device
    parents = torch.where(there, s["parents"][rows].long(), -1)
    tokens, u = s["drafts"][rows].long(), s["uniforms"][rows]
    lane, node, ids = torch.arange(lanes, device=dev), torch.arange(n, device=dev), torch.arange(v, device=dev)
    k = min(TOP_K, v) if c["sampled"] else 1
    cur = torch.zeros(lanes, dtype=torch.int64, device=dev)
    going = torch.ones(lanes, dtype=torch.bool, device=dev)
    accept = torch.zeros(lanes, dtype=torch.int64, device=dev)
    commits = torch.full((lanes, depth + 1), -1, device=dev)
    path = torch.full((lanes, depth + 1), -1, device=dev)
    path[:, 0] = 0
    for level in range(depth + 1):
        x = s["logits"][rows[lane, cur]]
        # larger values first, ties to the smaller id: the value's order above the id in one whole number
        raw = x.view(torch.int16).long()
        order = torch.where(raw < 0, -(raw + 32_768), raw) * v - ids
        best = torch.topk(order, k, dim=1).indices
        z = torch.gather(x, 1, best).double() / TEMPERATURE
        p = torch.exp(z - z[:, :1])
        p = p / p.sum(1, keepdim=True)
        kept = torch.cumsum(p, 1) - p < TOP_P
        p = torch.where(kept, p, 0.0)
        p = p / p.sum(1, keepdim=True)
        child = (parents == cur[:, None]) & (node > 0) & (level < depth)          # [lanes, n]
        same = best[:, None] == tokens[..., None]                                 # [lanes, n, k]
        before = (child[..., None] & same).long()
        gone = (torch.cumsum(before, 1) - before) > 0                             # tokens of the children before
        left = torch.where(gone, 0.0, p[:, None])
        total = left.sum(-1)
        yes = child & (u[..., 0] * total < torch.where(same, left, 0.0).sum(-1))
        taken = yes.any(1)
        to = yes.int().argmax(1)
        # the draw of a lane that stops here: from what its children leave
        rest = torch.where((child[..., None] & same).any(1), 0.0, p)
        run = torch.cumsum(rest, 1)
        over = (run > (u[lane, cur, 1] * rest.sum(1))[:, None]) & (rest > 0)
        spare = (rest > 0).int() * (1 + torch.arange(k, device=dev))
        pick = torch.where(over.any(1), over.int().argmax(1), spare.argmax(1))
        token = torch.where(taken, tokens[lane, to], best[lane, pick])
        commits[:, level] = torch.where(going, token, -1)
        going = going & taken
        accept += going
        cur = torch.where(going, to, cur)
        if level < depth:
            path[:, level + 1] = torch.where(going, to, -1)
    return accept.int(), commits.int(), path.int()


def _plain_commit(s):
    c = s["case"]
    lanes, p, depth = c["lanes"], c["page"], c["depth"]
    dev = s["path"].device
    ctx = (s["seq_lens"] - s["new_lens"]).long()
    lane, i = torch.arange(lanes, device=dev)[:, None], torch.arange(1, depth + 1, device=dev)
    moved = i <= s["accept"][:, None]
    source = ctx[:, None] + s["path"][:, 1:].long().clamp(min=0)
    target = (ctx[:, None] + i).expand(lanes, depth)
    last = s["block_table"].shape[1] - 1
    where = [(s["block_table"][lane, (x // p).clamp(max=last)].long()[moved], (x % p)[moved]) for x in (source, target)]
    (sp, so), (tp, to) = where
    if c["eight"]:
        kc, ks, vc, vs = s["caches"]
        for codes, scales in ((kc.view(torch.uint8), ks), (vc.view(torch.uint8), vs)):
            codes[tp, to] = codes[sp, so]
            scales[tp, :, to] = scales[sp, :, so]
    else:
        for x in s["caches"]:
            x[tp, to] = x[sp, so]
    s["context"].copy_(ctx + 1 + s["accept"])
    return s["caches"], s["context"]


def _plain_store(s):
    kept = s["slots"] >= 0
    slots, page = s["slots"][kept], s["case"]["page"]
    kc, ks, vc, vs = s["caches"]
    for codes, scales, x in ((kc, ks, s["k"]), (vc, vs, s["v"])):
        new, e = _quantise(x[kept])
        codes.view(torch.uint8)[slots // page, slots % page] = new.view(torch.uint8)
        scales[slots // page, :, slots % page] = e
    return s["caches"]


# ---- the definitions, in 64 bits --------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"attention": _exact_attention, "verify": _exact_verify, "commit": _exact_commit,
            "store": _exact_store}[case["op"]](case, s)


def _codes(dtype=torch.float64):
    """What the 256 codes of an 8-bit value stand for: sign, four bits of exponent, three of fraction."""
    def of(c):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        return math.nan if c & 127 == 127 else -x if c & 128 else x
    return torch.tensor([of(c) for c in range(256)], dtype=dtype, device="cuda")


def _exact_attention(case, s):
    p, group, d = case["page"], case["heads_q"] // case["heads_kv"], case["dim"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    value = _codes()
    words = _columns(case)
    masks, positions = [], []
    first = 0
    for lane, (parents, _, c) in enumerate(_trees(case)):
        n = len(parents)
        above = []                                    # of each node: itself and the nodes above it
        for i, parent in enumerate(parents):
            above.append({i} | (above[parent] if i else set()))
            masks.append([sum(1 << b for b in range(32) if w * 32 + b in above[i]) for w in range(words)])
            positions.append(c + len(above[i]) - 1)
        low = max(0, c - case["window"] + 1) // p if case["window"] else 0
        pages = s["block_table"][lane, low:-(-(c + n) // p)].long()
        where = torch.arange(low * p, low * p + pages.numel() * p, device="cuda")
        ok = (where < c).repeat(n, 1)
        if case["window"]:
            at = torch.tensor(positions[-n:], device="cuda")
            ok &= where > at[:, None] - case["window"]
        node = torch.tensor([[j in a for j in range(n)] for a in above], device="cuda")
        if case["window"] and not case["depth"]:
            i = torch.arange(n, device="cuda")
            node &= i > i[:, None] - case["window"]
        inside = (where >= c) & (where < c + n)
        ok[:, inside] = node[:, where[inside] - c]
        for h in range(case["heads_kv"]):
            if case["eight"]:
                kc, ks, vc, vs = s["caches"]
                keys, values = (value[x.view(torch.uint8)[pages, :, h].long()]
                                * torch.exp2(e[pages, h].double() - 127)[..., None] for x, e in ((kc, ks), (vc, vs)))
            else:
                keys, values = (x[pages, :, h].double() for x in s["caches"])
            keys, values = keys.reshape(-1, d), values.reshape(-1, d)
            for head in range(h * group, (h + 1) * group):
                w = s["q"][first:first + n, head].double() @ keys.T * s["scale"]
                w = torch.where(ok, w, -math.inf)
                total = torch.logsumexp(w, 1)
                out[first:first + n, head] = torch.exp(w - total[:, None]) @ values
                lse[first:first + n, head] = total
        first += n
    if not case["depth"]:
        return out, lse
    masks = torch.tensor(masks, dtype=torch.int64, device="cuda")
    return out, lse, torch.where(masks >= 1 << 31, masks - (1 << 32), masks).int(), _int32(positions)


def _exact_verify(case, s):
    v, depth = case["vocab"], case["depth"]
    drafts, uniforms = s["drafts"].tolist(), s["uniforms"].tolist()
    accept, commits, paths = [], [], []
    first = 0
    for parents, _, _ in _trees(case):
        cur, ids, path = 0, [], [0]
        while True:
            x = s["logits"][first + cur].double().cpu()
            level = torch.topk(x, min(v, TOP_K if case["sampled"] else 1)).values[-1]
            near = torch.nonzero(x >= level).flatten().tolist()
            near.sort(key=lambda t: (-float(x[t]), t))
            near = near[:TOP_K if case["sampled"] else 1]
            e = [math.exp((float(x[t]) - float(x[near[0]])) / TEMPERATURE) for t in near]
            total, run, q = math.fsum(e), 0.0, {}
            for t, y in zip(near, e):
                if run >= TOP_P:
                    break
                q[t] = y / total
                run += q[t]
            q = {t: y / math.fsum(q.values()) for t, y in q.items()}
            below = [i for i in range(1, len(parents)) if parents[i] == cur] if len(path) <= depth else []
            to = None
            for i in below:
                t = drafts[first + i]
                if uniforms[first + i][0] * math.fsum(q.values()) < q.get(t, 0.0):
                    to = i
                    break
                q.pop(t, None)
            if to is None:
                goal, run = uniforms[first + cur][1] * math.fsum(q.values()), 0.0
                for t, y in q.items():
                    run += y
                    if run > goal:
                        break
                ids.append(t)
                break
            ids.append(drafts[first + to])
            path.append(to)
            cur = to
        accept.append(len(path) - 1)
        commits.append(ids + [-1] * (depth + 1 - len(ids)))
        paths.append(path + [-1] * (depth + 1 - len(path)))
        first += len(parents)
    return _int32(accept), _int32(commits), _int32(paths)


def _exact_commit(case, s):
    p = case["page"]
    if case["eight"]:
        kc, ks, vc, vs = s["caches"]
        value = _codes()
        out = [value[kc.view(torch.uint8).long()], ks.clone(), value[vc.view(torch.uint8).long()], vs.clone()]
    else:
        out = [x.double() for x in s["caches"]]
    context = []
    table = s["block_table"].tolist()
    for lane, (_, path, c) in enumerate(_trees(case)):
        path = path[:case["depth"] + 1]
        place = lambda at: (table[lane][at // p], at % p)  # noqa: E731
        for i, node in enumerate(path):               # ascending: a later node is never where an earlier one went
            (tp, to), (sp, so) = place(c + i), place(c + node)
            for x in out:
                if x.dtype is torch.uint8:
                    x[tp, :, to] = x[sp, :, so].clone()
                else:
                    x[tp, to] = x[sp, so].clone()
        context.append(c + len(path))
    return out, _int32(context)


def _exact_store(case, s):
    page = case["page"]
    value = _codes()
    kc, ks, vc, vs = s["caches"]
    out = [value[kc.view(torch.uint8).long()], ks.clone(), value[vc.view(torch.uint8).long()], vs.clone()]
    kept = s["slots"] >= 0
    slots = s["slots"][kept]
    for at, x in ((0, s["k"]), (2, s["v"])):
        x = x[kept].double()
        largest = x.abs().amax(-1)
        # the exponents one after the other: the first whose 448 holds the vector
        e = torch.full(largest.shape, 7.0, dtype=torch.float64, device="cuda")
        for k in range(6, _least(s["k"].dtype) - 1, -1):
            e = torch.where(largest <= 448 * 2.0 ** k, float(k), e)
        y = (x / torch.exp2(e)[..., None]).clamp(-448, 448)
        step = torch.exp2((torch.frexp(y).exponent - 1).clamp(min=-6).double() - 3)   # three bits of fraction
        out[at][slots // page, slots % page] = torch.round(y / step) * step
        out[at + 1][slots // page, :, slots % page] = (e + 127).to(torch.uint8)
    return out
