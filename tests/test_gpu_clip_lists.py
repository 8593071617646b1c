"""What may happen to a gradient list around a call: dropped while another
stream still reads its table. What a table's memory is used for next here is
another valid table, whose tensors would show a call that reads it too early."""
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from gpu_util import device, say

pytestmark = pytest.mark.gpu


def _tensors(dev, seed, n=80, size=1700):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(size + i, generator=g).to(dev) for i in range(n)]


@pytest.mark.parametrize("current", [False, True])
def test_list_dropped_under_a_call_on_another_stream(current):
    dev = device()
    say("list dropped", current)
    grads = _tensors(dev, 1)
    outs = [torch.zeros_like(t) for t in grads]
    decoys = [torch.full_like(t, 5.0) for t in grads]
    glist, other = L.GradList(grads), L.GradList(decoys)
    norm, coef = torch.zeros(1, device=dev), torch.zeros(1, device=dev)
    L.logra_grad_clip(glist, 3.0, norm, coef, out=L.GradList(outs))
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream(device=dev)
    for _ in range(3):
        for t in outs:
            t.zero_()
        out = L.GradList(outs)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(5000000)
            if current:
                L.logra_grad_clip(glist, 3.0, norm, coef, out=out)
        if not current:
            L.logra_grad_clip(glist, 3.0, norm, coef, out=out, stream=side)
        del out
        later = [other.table.clone() for _ in range(8)]
        torch.cuda.synchronize()
        del later
        for got, ref, d in zip(outs, want, decoys):
            assert torch.equal(got, ref) and (d == 5.0).all()
