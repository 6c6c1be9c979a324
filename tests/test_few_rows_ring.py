"""The ring of factors of the few-rows form (8-bit cache): whatever the warps' timing, a key's factors are written over only
once the softmax of the tile that had them before has read them.  The order of the issuing warp and the teams' waits are
modelled here with the sources' constants, by themselves: no other wait is counted on.  No GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_draft_column_gb300", "csrc")


def read_early(pairs, stages, ahead, tiles=60):
    """Tiles whose factors may be gone before the softmax has read them."""
    # what the issuing warp has waited for when it issues each product: the softmax of tiles up to ...
    scores, weights, known = {}, {}, -1
    for i in range(min(ahead, tiles)):
        scores[i] = known
    for i in range(tiles):
        if i + ahead < tiles:
            scores[i + ahead] = known
        known = i                                # (the weights of tile i)
        weights[i] = known
    lost = set()
    for n in range(pairs, tiles):
        freed = n - 1 - stages // 2              # the tile whose product gave tile n - 1 its stage
        for issued in (scores, weights):
            if freed < 0 or issued[freed] < n - pairs:
                lost.add(n - pairs)
    return sorted(lost)


def test_the_model_sees_a_ring_that_is_too_short():
    assert read_early(5, 4, 1) == [] and read_early(6, 4, 2) == []
    assert read_early(4, 4, 1) and read_early(5, 4, 2) and read_early(5, 6, 1)


def test_factors_are_read_before_they_are_written_over():
    with open(os.path.join(CSRC, "attention.cuh")) as f:
        text = f.read()
    pairs = int(re.search(r"constexpr int kPairs = (\d+);", text)[1])
    ahead = int(re.search(r"static constexpr int kAhead = (\d+);", text)[1])
    stages = int(re.search(r"QT == 1 && D == 128 \? (\d+) : 3\)", text)[1])
    # the issuing warp goes by kAhead, and by nothing else
    assert "qk(i + S::kAhead)" in text and len(re.findall(r"\bqk\(", text)) == 2
    assert stages % 2 == 0 and read_early(pairs, stages, ahead) == []
