"""Many AdamW steps with moments in 8 bits beside the same with moments in 32.

What rounding by chance does to the mean over steps, with h the step of the codes
at a value (1/16 to 1/8 of it) and d what a step moves the value by, seen in
units of the block's scale:
  m: every rounding is unbiased, so m's is 0. Its deviation: h^2 / 4 a step at
     most, kept for 1 / (1 - beta1^2) steps: sqrt(m^2 / 256 / 0.19) = 0.15 |m|,
     and m is 0.23 of the gradient's deviation s (beta1 0.9): 0.034 s.
  v: the root's rounding is unbiased, so its square is too high by the rounding's
     variance: h |d| a step at most, kept for 1 / (1 - beta2) steps. d is
     (1 - beta2) / 2 |g^2 / v - 1| of the root from its own gradient and as
     much from that of the block's largest, which moves the scale; the mean of
     |g^2 / v - 1| is 0.97 of Gaussian gradients: between 0 and
     1/8 (0.97 + 0.97) / 2 = 0.121 of v. The root's deviation is the root of
     that, 0.35, and v's twice it.
Means over n elements are within 5 deviations / sqrt(n) of that."""
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from gpu_util import device

pytestmark = pytest.mark.gpu


def test_moments_over_many_steps():
    dev = device()
    blocks = 64
    n = 256 * blocks
    gen = torch.Generator(device=dev).manual_seed(1)
    size = torch.exp(0.5 * torch.randn(n, generator=gen, device=dev))
    grad = torch.zeros(n, device=dev)
    wide = L.AdamWList([torch.zeros(n, device=dev)], [grad])
    small = L.AdamWList([torch.zeros(n, device=dev)], [grad], state_bits=8)
    drift, high = [], []
    for step in range(1, 1001):
        grad.normal_(generator=gen).mul_(size)
        for lst in (wide, small):
            L.logra_adamw(lst, 1e-3, 0.9, 0.99, 1e-8, 0.0, step, seed=7)
        if step > 600 and step % 100 == 0:
            m, root = (t.float().reshape(blocks, 256) * s[:, None] for t, s in zip((small.exp_avg, small.exp_avg_sq), small.scales))
            drift.append(float(((m.reshape(n) - wide.exp_avg) / size).mean()))
            high.append(float((root.reshape(n) ** 2 / wide.exp_avg_sq).mean()))
    print("m: drift", drift, " v: ratio", high, flush=True)
    for d, h in zip(drift, high):
        assert abs(d) <= 5 * 0.034 / n ** 0.5
        assert -5 * 0.7 / n ** 0.5 <= h - 1 <= 0.121 + 5 * 0.7 / n ** 0.5
