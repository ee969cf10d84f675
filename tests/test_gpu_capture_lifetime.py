"""Objects that go away while a stream is capturing: the capture goes on, and
their handles are destroyed after it."""
import os
import sys

import pytest
import torch

ROOT = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["del", "close"])
@pytest.mark.parametrize("what", ["attn", "layer"])
def test_handles_dropped_in_a_capture(what, how):
    import decode_block as ex
    import serving_router_sigmoid_gb300 as moe
    x = torch.randn(64, 64, device="cuda")
    block = ex.Block(2, pages=8)
    gone, kept = vars(block).pop(what), block
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = x + 1
        if how == "close":
            gone.close()
        del gone
        y = y * 2
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, (x + 1) * 2)
    assert len(moe._parked) == 1
    moe.PagedAttention(1, 1, 1, 64).close()  # the next one to close takes it along
    assert not moe._parked
    if what == "layer":
        kept.attn.close()
    else:
        assert kept.layer.device_status() == 0
        kept.layer.close()
