"""The sketch over experts to the last bit, where arithmetic says what that is.

P = c s with s a sum of whole numbers below 2^24, so that every sum of its
terms is exact in fp32 in any order, and c = 1 / sqrt(r) a power of two (r = 64,
256): P is exact, with up to 24 significant bits. With one row per expert and
dY a power of two, S = dY P is one product; the three bf16 terms of P hold all
its bits (p0 its first 8, p1 the next, p2 the last), and p2 + p1 and
(p2 + p1) + p0 are exact in fp32. So S is dY P exactly. Two terms lose p2,
which the test sees to be there in over a quarter of the entries."""
import numpy as np
import pytest
import torch

import oracle
import rank_gradient_sketching_sketch_amd as L
from gpu_util import device, say

pytestmark = pytest.mark.gpu


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def _activations(T, k, seed):
    """Whole numbers that bf16 holds: half of them multiples of 2^12, half
    small, their magnitudes' sum below 2^24."""
    g = np.random.default_rng(seed)
    x = g.integers(-100, 101, (T, k)).astype(np.float64)
    x[:, ::2] *= 4096.0
    assert k <= 64 and np.abs(x).sum(1).max() < 2 ** 24 and (_bf16(x) == x).all()
    return x


@pytest.mark.parametrize("T,E,d,k,r", [
    (40, 40, 72, 64, 64),         # narrow projection, one row per expert
    (3, 3, 8, 56, 256),
    (200, 200, 136, 64, 256),     # the wide projection: more than 320 workgroups of the other
    (500, 1000, 16, 64, 256),     # half of the experts hold no row
])
@pytest.mark.parametrize("accumulate", [False, True])
def test_one_row_per_expert_is_exact(T, E, d, k, r, accumulate):
    dev = device()
    say("sketch experts exact", T, E, d, k, r, accumulate)
    x = _activations(T, k, T + r)
    g = np.random.default_rng(5)
    dy = 2.0 ** g.integers(-12, 4, (T, d)) * g.choice([-1.0, 1.0], (T, d))
    experts = np.sort(g.permutation(E)[:T])
    offsets = np.searchsorted(experts, np.arange(E + 1)).astype(np.int32)
    P = np.zeros((T, r))
    for t, e in enumerate(experts):
        A = oracle.sign_matrix(7, 2, 30 + int(e), r, k)     # +-c
        P[t] = A @ x[t]
    assert (P.astype(np.float32) == P).all()
    p0 = _bf16(P)
    p1 = _bf16(P - p0)
    p2 = _bf16(P - p0 - p1)
    assert (p0.astype(np.float64) + p1 + p2 == P).all() and (p2 != 0).mean() > 0.25
    S = torch.full((E, d, r), 0.0 if accumulate else float("nan"), device=dev)
    m = L.MatrixDesc(d, k, r, seed=7, step=2, matrix_id=30)
    L.logra_sketch_experts(m, torch.from_numpy(offsets).to(dev), torch.from_numpy(x).to(torch.bfloat16).to(dev),
                           torch.from_numpy(dy).to(torch.bfloat16).to(dev), S, accumulate)
    want = np.zeros((E, d, r))
    want[experts] = dy[:, :, None] * P[:, None, :]
    assert np.array_equal(S.cpu().double().numpy(), want)
