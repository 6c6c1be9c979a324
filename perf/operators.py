"""Cases of the paged-cache and logits operators: the plan of a step (block
tables and slot maps), the store of new keys and values, attention of the new
tokens over the paged cache, and the rules applied to target logits before
they are verified.

Every case is one step of a serving loop around speculative rounds: a batch of
lanes, each with some tokens already cached and a chunk of new ones (one token
when decoding, an anchor and its drafts when verifying, up to thousands while
a prompt is read).  Lengths follow from the case alone (its "pick"), values
from the seed.
"""
import math
import random

import torch

own = False

VOCAB = 248_046          # the target's output head
SHORTLIST = 131_072      # the shortlist head
WINDOW = 2_048           # the drafter's sliding window

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one lane decoding one token after a short prompt: the smallest step, where latency is what counts
        attention("decode 1x1", 1, 1, 1, 1_013, 1_013, 32, 8, 128, 16, "bf16", 0, 1),
        # eight lanes verifying an anchor and seven drafts over contexts of mixed lengths
        attention("verify 8x8", 8, 8, 8, 500, 16_000, 32, 8, 128, 64, "bf16", 0, 2),
        # one lane at the longest context, a block size of sixteen (anchor and fifteen drafts)
        attention("verify 1x16 at 262144", 1, 16, 16, 262_128, 262_128, 32, 8, 128, 128, "bf16", 0, 3),
        # a chunk of a long prompt
        attention("chunk 2048 at 30000", 1, 2_048, 2_048, 30_000, 30_000, 32, 8, 128, 64, "bf16", 0, 4),
        # a drafter's layer: a sliding window, half precision, small heads, ragged chunks over many lanes
        attention("drafter 64 lanes", 64, 1, 16, 100, 6_000, 16, 2, 64, 32, "f16", WINDOW, 5),
        # one lane, one column: plain sampling with penalties
        logits("logits 1x1", 1, 1, VOCAB, 0, 200, 0, 0.0, 1),
        # eight lanes of an anchor and seven drafts, penalties, a few biases, a grammar on some lanes
        logits("logits 8x8", 8, 8, VOCAB, 50, 4_000, 32, 0.5, 2),
        # many lanes at the largest block size, everything on
        logits("logits 64x16", 64, 16, VOCAB, 1_000, 16_000, 300, 1.0, 3),
        # the plan of a small verify step
        plan("plan 8x8", 8, 8, 8, 100, 20_000, 64, 1),
        # the plan of a large mixed step: decoding lanes among chunks of prompts
        plan("plan 1024 mixed", 1_024, 0, 512, 0, 60_000, 16, 2),
        # the new keys and values of a verify step
        store("store 8x8", 8 * 8, 8, 128, 64, 256, "bf16", 1),
        # those of a large batch of prompt chunks, some tokens without a page
        store("store 16384", 16_384, 8, 128, 16, 2_048, "bf16", 2),
    ]


def attention(name, lanes, new_lo, new_hi, ctx_lo, ctx_hi, heads_q, heads_kv, dim, page, dtype, window, pick):
    """Attention of each lane's new tokens over its cached ones and themselves."""
    return {"name": name, "op": "attention", "lanes": lanes, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "heads_q": heads_q, "heads_kv": heads_kv, "dim": dim, "page": page, "dtype": dtype,
            "window": window, "pick": pick}


def logits(name, lanes, cols, vocab, hist_lo, hist_hi, biases, masked, pick):
    """Penalties, biases and grammar masks on `cols` columns a lane; `masked`: the share of lanes with a grammar."""
    return {"name": name, "op": "logits", "lanes": lanes, "cols": cols, "vocab": vocab, "hist_lo": hist_lo,
            "hist_hi": hist_hi, "biases": biases, "masked": masked, "pick": pick}


def plan(name, lanes, new_lo, new_hi, ctx_lo, ctx_hi, page, pick):
    """Pages, block tables, positions and slots of a step's new tokens."""
    return {"name": name, "op": "plan", "lanes": lanes, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "page": page, "pick": pick}


def store(name, tokens, heads_kv, dim, page, pages, dtype, pick):
    """New keys and values into their slots of a paged cache."""
    return {"name": name, "op": "store", "tokens": tokens, "heads_kv": heads_kv, "dim": dim, "page": page,
            "pages": pages, "dtype": dtype, "pick": pick}


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    pick = rng.randrange(1 << 30)
    op = rng.choice(["attention", "attention", "attention", "logits", "logits", "plan", "store"])
    if op == "attention":
        dim = rng.choice([64, 128, 128, 256])
        heads_kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        page = rng.choice([16, 32, 64, 128])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        window = rng.choice([0, 0, 0, WINDOW, _log(rng, 64, 8_192)])
        kind = rng.choice(["decode", "verify", "verify", "chunk", "mixed"])
        if kind == "decode":
            lanes, new_lo, new_hi = _log(rng, 1, 64), 1, 1
        elif kind == "verify":
            lanes, new_lo, new_hi = _log(rng, 1, 64), 1, rng.randint(2, 16)
        elif kind == "chunk":
            lanes, new_hi = rng.randint(1, 3), _log(rng, 17, 2_048)
            new_lo = max(1, new_hi // 2)
        else:
            lanes, new_lo, new_hi = _log(rng, 4, 32), 0, _log(rng, 17, 512)
        # neither more keys than one lane at the longest context, nor more scores than the large chunk
        most = min(262_128, 4_000_000 // (lanes * heads_kv), 2_000_000_000 // (lanes * new_hi * heads_kv * group))
        ctx_hi = _log(rng, 40, max(64, most))
        return attention("", lanes, new_lo, new_hi, rng.choice([0, ctx_hi // 4, ctx_hi]), ctx_hi, heads_kv * group,
                         heads_kv, dim, page, dtype, window, pick)
    if op == "logits":
        lanes, cols = _log(rng, 1, 64), rng.choice([1, 1, 2, 4, 8, 16])
        vocab = rng.choice([VOCAB, VOCAB, SHORTLIST, _log(rng, 1_001, 248_045)])
        hist_hi = _log(rng, 1, 16_000)
        return logits("", lanes, cols, vocab, rng.choice([0, hist_hi // 2]), hist_hi, rng.choice([0, 0, 5, 300]),
                      rng.choice([0.0, 0.5, 1.0]), pick)
    if op == "plan":
        new_lo, new_hi = rng.choice([(0, _log(rng, 1, 512)), (1, 1), (8, 8), (1, 16)])
        lanes = _log(rng, 1, 1_024)
        return plan("", lanes, new_lo, new_hi, 0, _log(rng, 10, 60_000), rng.choice([16, 32, 64, 128]), pick)
    page = rng.choice([16, 32, 64, 128])
    heads_kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
    tokens = _log(rng, 1, 16_384 * 8 * 128 // max(8 * 128, heads_kv * dim))
    return store("", tokens, heads_kv, dim, page, -(-tokens * 2 // page) + 1, rng.choice(["bf16", "f16"]), pick)


# ---- lengths: from the case alone -------------------------------------------

def _lengths(case):
    """(new tokens, cached tokens) of each lane."""
    rng = random.Random(case["pick"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["lanes"])]
    new[rng.randrange(len(new))] = case["new_hi"]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["lanes"])]
    ctx[rng.randrange(len(ctx))] = case["ctx_hi"]
    return new, ctx


def _histories(case):
    """(prompt, whole history) lengths of each lane and which lanes have a grammar."""
    rng = random.Random(case["pick"])
    whole = [rng.randint(case["hist_lo"], case["hist_hi"]) for _ in range(case["lanes"])]
    whole[rng.randrange(len(whole))] = case["hist_hi"]
    prompt = [rng.randint(0, w) for w in whole]
    grammar = [rng.random() < case["masked"] for _ in whole]
    return prompt, whole, grammar


def work(case):
    if case["op"] == "attention":
        new, ctx = _lengths(case)
        w, g = case["window"] or 1 << 62, case["heads_q"] // case["heads_kv"]
        # keys in reach of the lane's first to last new token; (query, key) pairs under the causal mask
        keys = sum(c + n - max(0, c - w + 1) for n, c in zip(new, ctx) if n)
        pairs = sum(sum(min(c + t + 1, w) for t in range(n)) for n, c in zip(new, ctx))
        rows = sum(new) * case["heads_q"]
        pages = sum(-(-(c + n) // case["page"]) - max(0, c - w + 1) // case["page"] for n, c in zip(new, ctx) if n)
        return {"bytes": keys * case["heads_kv"] * case["dim"] * 4 + rows * (case["dim"] * 4 + 4) + 4 * pages
                + 8 * case["lanes"], "flops": 4 * pairs * case["heads_kv"] * g * case["dim"]}
    if case["op"] == "logits":
        _, whole, grammar = _histories(case)
        cols = case["lanes"] * case["cols"]
        masks = sum(grammar) * case["cols"] * -(-case["vocab"] // 32) * 4
        return {"bytes": cols * case["vocab"] * 4 + masks + 4 * sum(whole) + case["lanes"] * (20 + 8 * case["biases"])
                + 4 * (cols - case["lanes"]) + 4 * cols, "flops": 8 * cols * case["vocab"]}
    if case["op"] == "plan":
        new, ctx = _lengths(case)
        p = case["page"]
        pages = sum(max(0, -(-(c + n) // p) - -(-c // p)) for n, c in zip(new, ctx))
        touched = sum(-(-(c + n) // p) - c // p for n, c in zip(new, ctx) if n)
        return {"bytes": 24 * case["lanes"] + 8 * pages + 4 * touched + 12 * sum(new), "flops": 8 * sum(new)}
    kept = case["tokens"] - case["tokens"] // 16
    return {"bytes": kept * case["heads_kv"] * case["dim"] * 8 + 8 * case["tokens"], "flops": 0}


# ---- inputs -----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + case["pick"] % 999_983)
    s = {"case": case}
    {"attention": _prepare_attention, "logits": _prepare_logits, "plan": _prepare_plan,
     "store": _prepare_store}[case["op"]](case, g, s)
    if own:   # the handles that a program makes once, of its own buffers: pointers and sizes, no data
        _handles(case, s)
    return s


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _prepare_attention(case, g, s):
    new, ctx = _lengths(case)
    dt, p = _DTYPES[case["dtype"]], case["page"]
    need = [-(-(c + n) // p) for n, c in zip(new, ctx)]
    pages, most = sum(need) + 3, max(need)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((case["lanes"], most), dtype=torch.int32, device="cuda")
    at = 0
    for lane, n in enumerate(need):
        table[lane, :n] = perm[at:at + n]
        at += n
    shape = (pages, p, case["heads_kv"], case["dim"])
    s["k_cache"], s["v_cache"] = _normal(g, shape, dt), _normal(g, shape, dt)
    tokens = sum(new)
    s["q"] = _normal(g, (tokens, case["heads_q"], case["dim"]), dt)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["block_table"], s["cu_new"] = table, _int32(cu)
    s["new_lens"], s["seq_lens"] = _int32(new), _int32([c + n for n, c in zip(new, ctx)])
    s["scale"] = case["dim"] ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((tokens, case["heads_q"]), dtype=torch.float32, device="cuda")


def _prepare_logits(case, g, s):
    prompt, whole, grammar = _histories(case)
    lanes, cols, v = case["lanes"], case["cols"], case["vocab"]
    s["logits"] = (3 * _normal(g, (lanes * cols, v), torch.float32)).to(torch.bfloat16)
    # tokens of text repeat: ids fall off like a power law
    def ids(shape):
        return (v * torch.rand(shape, generator=g, device="cuda") ** 4).to(torch.int32).clamp_(0, v - 1)
    s["history"] = ids((lanes, case["hist_hi"]))
    s["prompt_lens"], s["history_lens"] = _int32(prompt), _int32(whole)
    s["drafts"] = ids((lanes, cols - 1)) if cols > 1 else None
    pen = torch.rand((lanes, 3), generator=g, device="cuda")
    s["penalties"] = (pen * torch.tensor([0.5, 1.0, 1.0], device="cuda")
                      + torch.tensor([1.0, 0.0, 0.0], device="cuda")).contiguous()
    s["bias_ids"] = s["bias_vals"] = s["bias_lens"] = s["mask"] = s["mask_rows"] = None
    if case["biases"]:
        nb = case["biases"]
        # distinct ids: a random start, then steps
        start = torch.randint(0, v, (lanes, 1), generator=g, device="cuda")
        s["bias_ids"] = ((start + torch.arange(nb, device="cuda") * (v // nb)) % v).to(torch.int32).contiguous()
        s["bias_vals"] = 5 * _normal(g, (lanes, nb), torch.float32)
        s["bias_lens"] = torch.full((lanes,), nb, dtype=torch.int32, device="cuda")
    if any(grammar):
        words = -(-v // 32)
        rows = sum(grammar) * cols
        # a grammar leaves few tokens: one word in two is empty, the others half full
        w = torch.randint(-(1 << 31), 1 << 31, (rows, words), generator=g, device="cuda")
        keep = torch.randint(0, 2, (rows, words), generator=g, device="cuda")
        s["mask"] = (w * keep).to(torch.int32)
        row, rs = 0, []
        for on in grammar:
            rs += list(range(row, row + cols)) if on else [-1] * cols
            row += cols if on else 0
        s["mask_rows"] = _int32(rs)
    s["out"] = torch.empty_like(s["logits"])


def _prepare_plan(case, g, s):
    new, ctx = _lengths(case)
    p = case["page"]
    held = [-(-c // p) for c in ctx]
    need = [-(-(c + n) // p) for n, c in zip(new, ctx)]
    most = max(need)
    pages = sum(need) + 16
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    h = torch.tensor(held, device="cuda")
    at = torch.cumsum(h, 0) - h
    i = torch.arange(most, device="cuda")
    where = at[:, None] + i
    s["table"] = torch.where(i < h[:, None], perm[where.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    s["free_pages"] = perm[sum(held):].contiguous()
    s["cursor"] = _int32([0])
    s["context_lens"], s["new_lens"], s["held"] = _int32(ctx), _int32(new), _int32(held)
    s["tokens"], s["lanes"], s["page"] = sum(new) + 5, case["lanes"], p   # a buffer a little larger than the step
    e32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    s["cu_new"], s["seq_lens"], s["held_out"], s["info"] = e32(s["lanes"] + 1), e32(s["lanes"]), e32(s["lanes"]), e32(4)
    s["positions"] = e32(s["tokens"])
    s["slots"] = torch.empty(s["tokens"], dtype=torch.int64, device="cuda")


def _prepare_store(case, g, s):
    dt = _DTYPES[case["dtype"]]
    shape = (case["pages"], case["page"], case["heads_kv"], case["dim"])
    s["k_cache"], s["v_cache"] = _normal(g, shape, dt), _normal(g, shape, dt)
    # a layer's projections give queries, keys and values side by side: keys and values are strided views
    t, h, d = case["tokens"], case["heads_kv"], case["dim"]
    kv = _normal(g, (t, 2 * h, d), dt)
    s["k"], s["v"] = kv[:, :h], kv[:, h:]
    slots = torch.randperm(case["pages"] * case["page"], generator=g, device="cuda")[:t]
    gone = torch.randperm(t, generator=g, device="cuda")[:t // 16]
    slots[gone] = -1
    s["slots"] = slots.to(torch.int64).contiguous()


# ---- the framework's operators ----------------------------------------------

def _handles(case, s):
    import speculative_decoding_draft_column_gb300 as sd
    if case["op"] in ("attention", "store"):
        s["cache"] = sd.PagedCache(s["k_cache"], s["v_cache"])
    if case["op"] == "attention":
        s["batch"] = sd.PagedBatch(s["block_table"], s["cu_new"], s["seq_lens"], page_size=case["page"])
        s["workspace"] = sd.new_attention_workspace()
    if case["op"] == "plan":
        s["batch"] = sd.PagedBatch(s["table"], s["cu_new"], s["seq_lens"], page_size=case["page"],
                                   context_lens=s["context_lens"], new_lens=s["new_lens"], held=s["held"],
                                   held_out=s["held_out"], positions=s["positions"], slots=s["slots"],
                                   info=s["info"])


def run(state):
    op = state["case"]["op"]
    return {"attention": _run_attention, "logits": _run_logits, "plan": _run_plan, "store": _run_store}[op](state)


def _run_attention(s):
    if own:
        import speculative_decoding_draft_column_gb300 as sd
        sd.spec_paged_attention(s["q"], s["cache"], s["batch"], s["scale"], s["out"], s["lse"], s["workspace"],
                                window=s["case"]["window"], max_new=s["case"]["new_hi"])
        return s["out"], s["lse"]
    return _plain_attention(s)


def _run_logits(s):
    if own:
        import speculative_decoding_draft_column_gb300 as sd
        c = s["case"]
        sd.spec_logits_process(s["logits"], c["lanes"], c["cols"], c["vocab"], s["out"], history=s["history"],
                               prompt_lens=s["prompt_lens"], history_lens=s["history_lens"], drafts=s["drafts"],
                               penalties=s["penalties"], bias_ids=s["bias_ids"], bias_vals=s["bias_vals"],
                               bias_lens=s["bias_lens"], mask=s["mask"], mask_rows=s["mask_rows"])
        return s["out"]
    return _plain_logits(s)


def _run_plan(s):
    if own:
        import speculative_decoding_draft_column_gb300 as sd
        sd.spec_paged_plan(s["batch"], s["free_pages"], s["cursor"])
        return [s[k] for k in ("table", "cu_new", "seq_lens", "held_out", "positions", "slots", "info")]
    return _plain_plan(s)


def _run_store(s):
    if own:
        import speculative_decoding_draft_column_gb300 as sd
        sd.spec_paged_store(s["k"], s["v"], s["slots"], s["cache"])
        return s["k_cache"], s["v_cache"]
    return _plain_store(s)


# ---- plain forms ------------------------------------------------------------

def _plain_attention(s):
    """All lanes at once, padded to the longest chunk and the longest context."""
    c = s["case"]
    lanes, hk, d = c["lanes"], c["heads_kv"], c["dim"]
    g, n, tokens = c["heads_q"] // hk, c["new_hi"], s["q"].shape[0]
    keys = s["block_table"].shape[1] * c["page"]
    dev = s["q"].device
    t = torch.arange(n, device=dev)
    at = s["cu_new"][:-1, None].long() + t                                     # [lanes, n] rows of q
    there = t < s["new_lens"][:, None]
    q = s["q"][at.clamp(max=tokens - 1)].float().view(lanes, n, hk, g, d).permute(0, 2, 3, 1, 4)
    pages = s["block_table"].long()
    k = s["k_cache"][pages].float().view(lanes, keys, hk, d).permute(0, 2, 3, 1)   # [lanes, hk, d, keys]
    v = s["v_cache"][pages].float().view(lanes, keys, hk, d).permute(0, 2, 1, 3)   # [lanes, hk, keys, d]
    x = torch.matmul(q.reshape(lanes, hk, g * n, d), k).mul_(s["scale"]).view(lanes, hk, g, n, keys)
    pos = (s["seq_lens"] - s["new_lens"])[:, None] + t                         # [lanes, n]
    j = torch.arange(keys, device=dev)
    hidden = j > pos[..., None]
    if c["window"]:
        hidden |= j <= pos[..., None] - c["window"]
    x.masked_fill_(hidden[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(lanes, hk, g * n, keys), v).view(lanes, hk, g, n, d) / z
    lse = (m + z.log()).squeeze(-1)
    rows = at[there]
    s["out"][rows] = o.permute(0, 3, 1, 2, 4).reshape(lanes, n, hk * g, d)[there].to(s["out"].dtype)
    s["lse"][rows] = lse.permute(0, 3, 1, 2).reshape(lanes, n, hk * g)[there]
    return s["out"], s["lse"]


def _plain_logits(s):
    c = s["case"]
    lanes, cols, v = c["lanes"], c["cols"], c["vocab"]
    x = s["logits"].float().view(lanes, cols, v)
    h = s["history"].long()
    i = torch.arange(h.shape[1], device=h.device)
    said = ((i >= s["prompt_lens"][:, None]) & (i < s["history_lens"][:, None])).float()
    asked = (i < s["prompt_lens"][:, None]).float()
    count = torch.zeros((lanes, v), device=h.device).scatter_add_(1, h, said)[:, None]
    seen = torch.zeros((lanes, v), device=h.device).scatter_add_(1, h, asked)[:, None] > 0
    if cols > 1:
        # column j counts the drafts before it
        d = s["drafts"].long()
        before = (torch.arange(cols, device=h.device)[:, None] > torch.arange(cols - 1, device=h.device)).float()
        more = torch.zeros((lanes, cols, v), device=h.device)
        more.scatter_add_(2, d[:, None].expand(lanes, cols, cols - 1).contiguous(),
                          before.expand(lanes, cols, cols - 1).contiguous())
        count = count + more
    r, f, p = (s["penalties"][:, k, None, None] for k in range(3))
    x = torch.where(seen | (count > 0), torch.where(x > 0, x / r, x * r), x)
    x = x - (f * count + p * (count > 0))
    if s["bias_ids"] is not None:
        x = x + torch.zeros((lanes, v), device=h.device).scatter_add_(1, s["bias_ids"].long(), s["bias_vals"])[:, None]
    x = x.view(lanes * cols, v)
    if s["mask"] is not None:
        t = torch.arange(v, device=h.device)
        bits = (s["mask"][:, t // 32] >> (t % 32)) & 1
        row = s["mask_rows"].long()
        x = x.masked_fill((bits[row.clamp(min=0)] == 0) & (row >= 0)[:, None], float("-inf"))
    return x.to(torch.bfloat16)


def _plain_plan(s):
    p, most, dev = s["page"], s["table"].shape[1], s["table"].device
    new, ctx, held = s["new_lens"].long(), s["context_lens"].long(), s["held"].long()
    seq = ctx + new
    need = (seq + p - 1) // p
    want = (need.clamp(max=most) - held).clamp(min=0)
    upto = torch.cumsum(want, 0)
    first = upto - want
    free = s["free_pages"].numel() - s["cursor"].long()
    got = torch.minimum((free - first).clamp(min=0), want)
    i = torch.arange(most, device=dev)
    fresh = (i >= held[:, None]) & (i < (held + got)[:, None])
    source = s["cursor"].long() + first[:, None] + i - held[:, None]
    pages = s["free_pages"][source.clamp(0, s["free_pages"].numel() - 1)]
    table = torch.where(fresh, pages, s["table"])
    held_out = held + got
    ends = torch.cumsum(new, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), ends])
    t = torch.arange(s["tokens"], device=dev)
    lane = torch.searchsorted(ends, t, right=True)
    there = lane < s["lanes"]
    lane = lane.clamp(max=s["lanes"] - 1)
    pos = ctx[lane] + t - cu[lane]
    page = pos // p
    slots = table[lane, page.clamp(0, most - 1)].long() * p + pos % p
    slots = torch.where(there & (page < held_out[lane]), slots, -1)
    info = torch.stack([ends[-1], s["cursor"][0] + got.sum(), (want - got).sum(), (need > most).sum()])
    return [table, cu.int(), seq.int(), held_out.int(), torch.where(there, pos, 0).int(), slots, info.int()]


def _plain_store(s):
    kept = s["slots"] >= 0
    slots = s["slots"][kept]
    s["k_cache"].view(-1, *s["k_cache"].shape[2:])[slots] = s["k"][kept]
    s["v_cache"].view(-1, *s["v_cache"].shape[2:])[slots] = s["v"][kept]
    return s["k_cache"], s["v_cache"]


# ---- the definitions, in 64 bits --------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"attention": _exact_attention, "logits": _exact_logits, "plan": _exact_plan,
            "store": _exact_store}[case["op"]](case, s)


def _exact_attention(case, s):
    new, ctx = _lengths(case)
    p, group = case["page"], case["heads_q"] // case["heads_kv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for lane, (n, c) in enumerate(zip(new, ctx)):
        if n == 0:
            continue
        low = max(0, c - case["window"] + 1) // p if case["window"] else 0
        pages = s["block_table"][lane, low:-(-(c + n) // p)].long()
        where = torch.arange(low * p, low * p + pages.numel() * p, device="cuda")
        at = torch.arange(c, c + n, device="cuda")[:, None]
        ok = where <= at
        if case["window"]:
            ok &= where > at - case["window"]
        for h in range(case["heads_kv"]):
            keys = s["k_cache"][pages, :, h].double().reshape(-1, case["dim"])
            values = s["v_cache"][pages, :, h].double().reshape(-1, case["dim"])
            for head in range(h * group, (h + 1) * group):
                w = s["q"][first:first + n, head].double() @ keys.T * s["scale"]
                w = torch.where(ok, w, -math.inf)
                total = torch.logsumexp(w, 1)
                out[first:first + n, head] = torch.exp(w - total[:, None]) @ values
                lse[first:first + n, head] = total
        first += n
    return out, lse


def _exact_logits(case, s):
    prompt, whole, _ = _histories(case)
    out = s["logits"].double()
    cols, v = case["cols"], case["vocab"]
    pen = s["penalties"].double().tolist()
    for lane in range(case["lanes"]):
        h = s["history"][lane].long()
        asked = torch.bincount(h[:prompt[lane]], minlength=v)
        said = torch.bincount(h[prompt[lane]:whole[lane]], minlength=v)
        bias = torch.zeros(v, dtype=torch.float64, device="cuda")
        if s["bias_ids"] is not None:
            bias[s["bias_ids"][lane].long()] = s["bias_vals"][lane].double()
        r, f, p = pen[lane]
        for j in range(cols):
            if j:
                said[int(s["drafts"][lane, j - 1])] += 1
            x = out[lane * cols + j]
            met = (asked + said) > 0
            x[met] = torch.where(x[met] > 0, x[met] / r, x[met] * r)
            x -= f * said
            x[said > 0] -= p
            x += bias
            if s["mask"] is not None and int(s["mask_rows"][lane * cols + j]) >= 0:
                words = s["mask"][int(s["mask_rows"][lane * cols + j])]
                allowed = torch.stack([(words >> b) & 1 for b in range(32)], 1).reshape(-1)[:v]
                x[allowed == 0] = -math.inf
    return out


def _exact_plan(case, s):
    new, ctx = _lengths(case)
    p = case["page"]
    table, free = s["table"].tolist(), s["free_pages"].tolist()
    held, most = s["held"].tolist(), s["table"].shape[1]
    cu, seq, positions, slots, used, short, over = [0], [], [], [], 0, 0, 0
    for lane, (n, c) in enumerate(zip(new, ctx)):
        need = -(-(c + n) // p)
        over += need > most
        while held[lane] < min(need, most):
            if used == len(free):
                short += min(need, most) - held[lane]
                break
            table[lane][held[lane]] = free[used]
            used += 1
            held[lane] += 1
        for at in range(c, c + n):
            positions.append(at)
            slots.append(table[lane][at // p] * p + at % p if at // p < held[lane] else -1)
        cu.append(cu[-1] + n)
        seq.append(c + n)
    info = [cu[-1], used, short, over]
    positions += [0] * (s["tokens"] - len(positions))
    slots += [-1] * (s["tokens"] - len(slots))
    return [_int32(table), _int32(cu), _int32(seq), _int32(held), _int32(positions),
            torch.tensor(slots, dtype=torch.int64, device="cuda"), _int32(info)]


def _exact_store(case, s):
    page = case["page"]
    k, v = s["k_cache"].double(), s["v_cache"].double()
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            k[slot // page, slot % page] = s["k"][t].double()
            v[slot // page, slot % page] = s["v"][t].double()
    return k, v
