"""Zeros keep their sign as codes, whatever the scales of the blocks beside them:
an element's code hangs on its block alone. Codes and scales: equal, bit by bit."""
import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from oracle import layers as ox
from gpu_util import device

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _check(x, block_rows, turned=False):
    dev = device()
    n, k = x.shape
    shape = (k, n) if turned else (n, k)
    grid = (-(-n // block_rows), -(-k // 128))
    codes = torch.zeros(shape, dtype=torch.uint8, device=dev).view(F8)
    scales = torch.zeros(grid[::-1] if turned else grid, device=dev)
    L.logra_fp8_quantize(x.to(dev), codes, scales, block_rows=block_rows, transpose=turned)
    want, ws = ox.quantize(x.float().numpy(), block_rows, turned)
    got = codes.view(torch.uint8).cpu().numpy()
    assert np.array_equal(got, want) and np.array_equal(scales.cpu().numpy(), ws)
    return got


def _rows(dt, n, k):
    x = torch.randn(n, k, generator=torch.Generator().manual_seed(n + k))
    x[:, ::3] = -0.0
    x[:, 1::6] = 0.0
    x[:, 2::9] = -1e-30                     # quotients that vanish keep their sign too
    return x.to(dt)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows(dt):
    x = _rows(dt, 13, 300)
    alone = _check(x, 1)
    assert (alone[:, ::3] == 0x80).all() and (alone[:, 1::6] == 0).all()
    y = torch.zeros(13, 300, dtype=dt)
    y[0], y[1], y[4], y[12] = 1e-30, 1e30, -0.0, 1e38
    both = torch.stack([x, y], 1).reshape(26, 300)      # every row beside one of another size
    assert np.array_equal(_check(both, 1)[::2], alone)


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_tiles(dt, turned):
    x = _rows(dt, 200, 300)
    x[128:, 128:256] *= 1e-30
    x[:128, 256:] = -0.0                    # a block of nothing else
    got = _check(x, 128, turned)
    got = got.T if turned else got
    assert (got[:, ::3] == 0x80).all() and (got[:128, 256:] == 0x80).all()
