"""An element's update hangs on the element alone, to the last bit: not on what the
moments beside it are, though very small and very large ones take another way to
their roots."""
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("far", [2.0 ** -120, 2.0 ** 110])
def test_roots(far):
    dev = device()
    n = 1 << 24                                 # all fp32 values of two binades
    v = (torch.arange(n, dtype=torch.int32, device=dev) + (127 << 23)).view(torch.float32)
    out = []
    for other in (False, True):
        # p' = -g / root of v: the root's last bit shows in nearly all of them
        p, g = torch.zeros(n, device=dev), torch.full((n,), 2.0 ** -40, device=dev)
        state = [torch.zeros(n, device=dev), v.clone()]
        if other:
            state[1][::256] = far
        lst = L.AdamWList([p], [g], state=state)
        L.logra_adamw(lst, 1.0, 0.0, 0.5, 0.0, 0.0, 200)
        out.append(p.reshape(-1, 256)[:, 1:])
    differ = int((out[0] != out[1]).sum())
    assert differ == 0 and bool(torch.isfinite(out[0]).all())
