"""The layer's router is bf16: another type is refused, not read as if it were; the example decodes with the router that
it balanced."""
import importlib.util
import os

import pytest
import torch


def test_layer_refuses_other_router_types():
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300 as M
    pool = torch.zeros(16, 3 * 256 * 128, dtype=torch.bfloat16)
    for dtype in (torch.float32, torch.float16):
        with pytest.raises(ValueError, match="w_router"):
            M.SlotCachedMoELayer(torch.zeros(256, 16, dtype=dtype), pool, 2, 128, M.MODE_RESIDENT)


@pytest.mark.gpu
def test_the_example_routes_by_its_balanced_router():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "w4_layer.py")
    spec = importlib.util.spec_from_file_location("w4_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    r = ex.main(["--tokens", "4", "--steps", "20"])
    for t in range(16):
        x = r["embed"][t:t + 1]
        res = r["layer"].forward(x)
        logits = (x.double() @ r["router"].double())[0]
        want = torch.topk(logits, ex.K)
        if float(want.values[-1] - logits.sort(descending=True).values[ex.K]) < 1e-4:
            continue  # fp32 sums may order these two the other way
        assert sorted(res["ids"][0].tolist()) == sorted(want.indices.tolist())
        w = torch.softmax(logits[res["ids"][0].long()], 0)
        assert torch.allclose(res["w"][0].double(), w, atol=1e-5)
        assert bool(res["out"].isfinite().all())
