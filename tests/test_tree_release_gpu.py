"""Verify of trees on one host thread while another releases the library's scratch: a call holds the scratch until it is
launched, and the release waits for what was launched.  Needs a GPU."""
from __future__ import annotations

import threading

import numpy as np
import pytest

from tests import tree_ref as ref
from tests.test_tree_gpu import _i32, _verify_case

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


def test_release_while_trees_are_verified(sd):
    import torch
    rng = np.random.default_rng(11)
    cu, logits, drafts, parents = _verify_case(rng, [6, 3], 5_000, 4)
    want = list(ref.verify(logits.double().cpu().numpy(), drafts.tolist(), parents, cu, 4)[:3])
    d, p, c = _i32(drafts.tolist()), _i32(parents), _i32(cu)
    torch.cuda.synchronize()
    errors, done = [], threading.Event()

    def verify():
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    got = sd.tree_verify(logits, d, p, c, 4)
                    if [x.tolist() for x in got] != want:
                        errors.append("differs from the plain form")
        except Exception as e:                          # noqa: BLE001 - reported below
            errors.append(repr(e))
        finally:
            done.set()

    def release():
        try:
            torch.cuda.set_device(0)
            while not done.wait(1e-3):
                sd.spec_release()
        except Exception as e:                          # noqa: BLE001 - reported below
            errors.append(repr(e))

    ts = [threading.Thread(target=verify), threading.Thread(target=release)]
    for t in ts:
        t.start()
    for t in ts:
        t.join(timeout=300)
    assert not any(t.is_alive() for t in ts) and not errors, errors[:3]
    assert sd.spec_device_status() is None
