"""A serving loop of speculative rounds over a paged cache, on a toy target.

    python examples/paged_round.py

The target is one attention layer whose queries, keys and values depend on the
token alone (tables, no positions), under a random output head; the drafter is a
table of likely next tokens.  What is real is everything around it: a step is

    spec_paged_plan        pages, positions and slots of the new tokens
    spec_paged_store       their keys and values into the cache
    spec_paged_attention   over the cached and the new tokens, causal
    spec_logits_process    penalties for what was said, a grammar's mask
    spec_verify            drafts against the target's argmax, commits

and the lengths stay on the device from step to step: a rejected draft's keys are
overwritten by the next step's, its pages stay with the lane.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

VOCAB, HEADS_Q, HEADS_KV, DIM, PAGE = 4_096, 8, 2, 64, 16


class Toy:
    """The toy target and drafter: tables made from a seed."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *n: torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.q, self.k, self.v = r(VOCAB, HEADS_Q, DIM), r(VOCAB, HEADS_KV, DIM), r(VOCAB, HEADS_KV, DIM)
        self.head = r(HEADS_Q * DIM, VOCAB)
        self.likely = torch.randint(0, VOCAB, (VOCAB,), generator=g, device="cuda", dtype=torch.int32)
        # a grammar that allows three tokens in four
        bits = torch.rand((VOCAB // 32, 32), generator=g, device="cuda") < 0.75
        self.allowed = bits.flatten()
        weight = torch.tensor([1 << b for b in range(31)] + [-(1 << 31)], dtype=torch.int64, device="cuda")
        self.mask = (bits * weight).sum(1).to(torch.int32).view(1, -1)


def generate(lanes=4, rounds=8, gamma=7, seed=0):
    import speculative_decoding_draft_column_gb300 as sd
    toy = Toy(seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    width = gamma + 1
    prompt = torch.randint(5, 40, (lanes,), generator=g, device="cuda", dtype=torch.int32)
    longest = int(prompt.max())
    room = longest + (rounds + 1) * width + 1
    history = torch.randint(0, VOCAB, (lanes, room), generator=g, device="cuda", dtype=torch.int32)
    said = prompt.clone()                                        # tokens of history in use
    pages = lanes * (room // PAGE + 2)
    # twice the pages the lanes need, in any order, and whatever was in them
    cache = sd.PagedCache(*(torch.full((2 * pages, PAGE, HEADS_KV, DIM), float("nan"), dtype=torch.bfloat16, device="cuda")
                            for _ in range(2)))
    free = torch.randperm(2 * pages, generator=g, device="cuda").to(torch.int32)
    cursor = torch.zeros(1, dtype=torch.int32, device="cuda")
    # penalties: repetition 1.1, and a presence penalty that rules out saying a token twice
    penalties = torch.tensor([[1.1, 0.2, 1e4]], device="cuda").expand(lanes, 3).contiguous()
    workspace = sd.new_attention_workspace()
    rows = torch.arange(lanes, device="cuda")

    def step(batch, tokens, max_new):
        """Attention of the batch's new tokens (a flat list), their keys and values stored on the way."""
        sd.spec_paged_plan(batch, free, cursor)
        ids = tokens.long()
        sd.spec_paged_store(toy.k[ids], toy.v[ids], batch.slots, cache)
        out, _ = sd.paged_attention(toy.q[ids], cache, batch, max_new=max_new, workspace=workspace)
        cursor.copy_(batch.info[1:2])
        return out

    def logits_of(out):
        return (out.reshape(-1, HEADS_Q * DIM) @ toy.head * 0.2).to(torch.bfloat16)

    def rules(cols, drafts=None):
        return dict(history=history, prompt_lens=prompt, history_lens=said, penalties=penalties, drafts=drafts, mask=toy.mask,
                    mask_rows=torch.zeros(lanes * cols, dtype=torch.int32, device="cuda"))

    # the prompts: one chunk a lane, all but the last token, which is the first anchor
    fill = sd.PagedBatch.create(lanes, room // PAGE + 2, int(prompt.sum()) - lanes, PAGE)
    fill.new_lens.copy_(prompt - 1)
    chunk = torch.cat([history[lane, :int(n) - 1] for lane, n in enumerate(prompt)])
    step(fill, chunk, longest)

    # the rounds: the anchor and the drafts after it
    batch = sd.PagedBatch.create(lanes, fill.max_pages, lanes * width, PAGE)
    batch.block_table.copy_(fill.block_table)
    batch.context_lens.copy_(fill.seq_lens)
    batch.held.copy_(fill.held_out)
    batch.new_lens.fill_(width)
    accepted = []
    for _ in range(rounds):
        anchor = history[rows, said.long() - 1]
        drafts = [toy.likely[anchor.long()]]
        for _ in range(gamma - 1):
            drafts.append(toy.likely[drafts[-1].long()])
        drafts = torch.stack(drafts, 1).contiguous()
        out = step(batch, torch.cat([anchor[:, None], drafts], 1).reshape(-1), width)
        raw = logits_of(out)
        # the toy's drafter is right about half the time: lift its next token's logit
        lift = raw.view(lanes, width, VOCAB)
        lift[:, :gamma].scatter_add_(2, drafts.long()[:, :, None], (torch.rand((lanes, gamma, 1), generator=g, device="cuda") < 0.6).to(raw.dtype) * 40)
        target = sd.process_logits(raw, lanes, width, **rules(width, drafts))
        acc, commits = sd.verify(target, drafts)
        # the commits into the history; the anchor and the accepted drafts are cached
        at = said.long()[:, None] + torch.arange(width, device="cuda")
        history.scatter_(1, at, torch.where(commits >= 0, commits, history.gather(1, at)))
        said += acc + 1
        batch.context_lens += acc + 1
        batch.held.copy_(batch.held_out)
        accepted.append(acc)
    return {"sd": sd, "toy": toy, "cache": cache, "batch": batch, "history": history, "said": said, "prompt": prompt,
            "accepted": torch.stack(accepted), "last_target": target, "last_commits": commits}


if __name__ == "__main__":
    r = generate()
    torch.cuda.synchronize()
    r["sd"].spec_device_status()
    for lane in range(r["said"].numel()):
        p, s = int(r["prompt"][lane]), int(r["said"][lane])
        print(f"lane {lane}: prompt of {p}, {s - p} tokens in {r['accepted'].shape[0]} rounds "
              f"(accepted {r['accepted'][:, lane].tolist()}): {r['history'][lane, p:s].tolist()}")
