"""The example's loop: the pieces fit, every rank holds the same 4-bit weight, and it learns."""
import importlib.util
import os

import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sharded_update_learns():
    spec = importlib.util.spec_from_file_location("sharded_update", os.path.join(ROOT, "examples", "sharded_update.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    t = example.Trainer(ranks=4, n=256, k=160, batch=128)
    first = float(t.step())
    for _ in range(150):
        last = t.step()
    say("sharded update", first, float(last))
    assert float(last) < 0.2 * first and int(t.ctrl.step) == 151
    whole = torch.cat([c.view(-1, t.k) for c in t.copies])
    want = dps.dp_mxfp4_quantize(whole)
    for w in t.weights:
        assert torch.equal(w.codes, want.codes)
        assert torch.equal(dps.dp_mxfp4_dequantize(w), dps.dp_mxfp4_dequantize(want))
    assert all(torch.equal(c, p.bfloat16()) for c, p in zip(t.copies, t.params))
