"""Products over experts whose offsets decrease somewhere: rows that no expert has
and what lies behind Y stay, and an element of a row that some have gets the
product of one of them or stays (a kernel may have workgroups for as many tiles
alone as offsets that do not decrease can have: M / 16 + the experts, times those
of the features; these have more).
Codes are small whole numbers and scales 1: exact."""
import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from gpu_util import device, say

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,n,k", [(50, 40, 32), (900, 300, 272)])
def test_decreasing(M, n, k, dt):
    dev = device()
    say("decreasing offsets", M, n, k, dt)
    g = torch.Generator().manual_seed(M)
    E, kb = 5, -(-k // 128)
    off = [0, M * 4 // 5, M // 5, M // 5, M * 9 // 10, -7]
    x = torch.randint(-2, 3, (M, k), generator=g).float()
    w = torch.randint(-2, 3, (E, n, k), generator=g).float()
    y = torch.full((M + 8, n), 0.5, dtype=dt, device=dev)
    L.logra_fp8_matmul(x.to(F8).to(dev), torch.ones(M, kb, device=dev), w.to(F8).to(dev), torch.ones(E, -(-n // 128), kb, device=dev),
                       y[:M], offsets=torch.tensor(off, dtype=torch.int32, device=dev))
    got = y.double().cpu().numpy()
    ref = np.zeros((E, M + 8, n))
    ref[:, :M] = torch.einsum("mk,enk->emn", x.double(), w.double()).to(dt).double().numpy()
    has = np.zeros((E, M + 8), bool)
    for e in range(E):
        a, b = max(off[e], 0), min(max(off[e + 1], 0), M)
        has[e, a:max(a, b)] = True
    for r in range(M + 8):
        fits = got[r] == 0.5                                    # products are whole numbers
        for e in np.flatnonzero(has[:, r]):
            fits |= got[r] == ref[e][r]
        assert fits.all(), r
    assert (got[:M] != 0.5).any()
