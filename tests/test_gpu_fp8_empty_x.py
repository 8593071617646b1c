"""Products over experts where x has no rows, or the order names none that it has:
every row of Y that an expert has is zeros, the others stay."""
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from gpu_util import device, say

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,n,k", [(5, 40, 32), (200, 300, 144), (700, 260, 2064), (3000, 384, 1040)])
@pytest.mark.parametrize("rows", [0, 1])
def test_rows_that_are_not_there(rows, M, n, k, dt):
    dev = device()
    say("empty x", rows, M, n, k, dt)
    E, kb = 3, -(-k // 128)
    w = torch.randn(E, n, k, generator=torch.Generator().manual_seed(1)).to(F8).to(dev)
    ws = torch.ones(E, -(-n // 128), kb, device=dev)
    x, xs = torch.ones(rows, k, device=dev).to(F8), torch.ones(rows, kb, device=dev)
    offsets = torch.tensor([0, M // 3, M // 3, M - 1], dtype=torch.int32, device=dev)
    order = torch.arange(M, dtype=torch.int32, device=dev) + rows
    y = torch.full((M, n), 7.0, dtype=dt, device=dev)
    L.logra_fp8_matmul(x, xs, w, ws, y, offsets=offsets, order=order, topk=1)
    assert not y[:M - 1].any() and bool((y[M - 1] == 7).all())
