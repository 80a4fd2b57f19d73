"""The example that runs the 4-bit layer, the balance loss and the 4-bit head together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_w4_layer_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "w4_layer.py")
    spec = importlib.util.spec_from_file_location("w4_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    r = ex.main(["--tokens", "8", "--steps", "40"])
    assert r["after"][0] < r["before"][0] and r["after"][1] < r["before"][1]
    assert len(r["text"]) == 8 and all(0 <= t < ex.VOCAB for t in r["text"])
    assert r["packed"].nbytes < 0.3 * r["slabs"].nbytes
    # the head is the quantised matrix: a 4-bit step of a group's largest element is an eighth of it
    x = torch.eye(ex.H, device="cuda", dtype=torch.bfloat16)[:32]
    y = torch.cat([r["op_head"].forward(row) for row in x.split(1)])
    w = r["head"][:32].float()
    top = r["head"][:ex.GROUP].float().abs().amax(0)
    assert bool(((y - w).abs() <= top * (0.125 * 1.01)).all())
