"""Column slices of one buffer as the parameters (and copies) of a list: bit by bit
what the same tensors give by themselves, and what lies between them stays."""
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_slices(bits):
    dev = device()
    g = torch.Generator().manual_seed(2)
    rows, cuts = 70, [(0, 33), (33, 64), (65, 300)]
    wide = torch.randn(rows, 301, generator=g).to(dev)
    low = torch.zeros(rows, 301, dtype=torch.bfloat16, device=dev)
    start = wide.clone()
    slices, copies = [wide[:, a:b] for a, b in cuts], [low[:, a:b] for a, b in cuts]
    alone, cop = [s.clone() for s in slices], [c.clone() for c in copies]
    grads = [torch.randn(rows, b - a, generator=g).to(dev) for a, b in cuts]
    one = L.AdamWList(slices, grads, state_bits=bits, copies=copies)
    two = L.AdamWList(alone, [d.clone() for d in grads], state_bits=bits, copies=cop)
    for step in (1, 2, 3):
        for lst in (one, two):
            L.logra_adamw(lst, 1e-2, 0.9, 0.99, 1e-8, 0.1, step, seed=4)
    for s, c, a, d in zip(slices, copies, alone, cop):
        assert torch.equal(s, a) and torch.equal(c, d) and not torch.equal(c, torch.zeros_like(c))
    assert torch.equal(wide[:, 64], start[:, 64]) and torch.equal(wide[:, 300], start[:, 300])
    assert not low[:, 64].any() and not low[:, 300].any()
    with pytest.raises(L.LograError):
        L.AdamWList([wide[:, :34], wide[:, 33:64]], [grads[0].new_zeros(rows, 34), grads[1]])
