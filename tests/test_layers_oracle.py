"""The plain forms of routing, 8-bit codes and AdamW against their own
definitions, by other means: gradients by differences, codes against torch's
own conversion, the rounding by chance on average. No GPU."""
import numpy as np
import pytest
import torch

from oracle import layers as ox


@pytest.mark.parametrize("score", [ox.SOFTMAX, ox.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_is_the_weights_slope(score, renorm):
    g = np.random.default_rng(3)
    x = g.normal(size=(5, 9))
    ids, _ = ox.route(x, 4, score, renormalize=renorm)
    ids[1, 2], ids[2] = -1, [3, 3, 40, 0]           # a choice that is none, one expert twice, one that is not there
    dw = g.normal(size=ids.shape)
    got, _ = ox.route_backward(x, ids, dw, score, renorm, 1.7)
    h = 1e-6
    for t in range(5):
        for e in range(9):
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            d = ((ox.route_weights(up, ids, score, renorm, 1.7) - ox.route_weights(down, ids, score, renorm, 1.7)) * dw).sum()
            assert abs(d / (2 * h) - got[t, e]) < 1e-8          # h^2 / 6 of a third derivative of order one, and rounding 1e-16 / h


def test_route_groups_against_a_search():
    g = np.random.default_rng(5)
    x, bias = g.normal(size=(40, 24)), 0.2 * g.normal(size=24)
    ids, _ = ox.route(x, 3, ox.SIGMOID, bias=bias, groups=6, topk_groups=2, group_best=2)
    key = 1 / (1 + np.exp(-x)) + bias
    for t in range(40):
        rank = [sum(sorted(key[t, 4 * i:4 * i + 4])[-2:]) for i in range(6)]
        kept = sorted(range(6), key=lambda i: -rank[i])[:2]
        pool = [(key[t, e], -e) for i in kept for e in range(4 * i, 4 * i + 4)]
        assert list(ids[t]) == [-e for _, e in sorted(pool, reverse=True)[:3]]


def test_codes_are_torchs():
    v = np.arange(256).astype(np.uint8)
    mine, torchs = ox.decode(v), torch.from_numpy(v).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(mine, torchs, equal_nan=True)
    g = np.random.default_rng(0)
    q = np.concatenate([g.normal(size=4000) * 10.0 ** g.uniform(-4, 2.6, 4000), [0.0, -0.0, 448.0, -448.0, 17.0, 0.001, np.nan]])
    q = np.clip(q, -448, 448).astype(np.float32)
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = ox.encode(q)
    assert np.array_equal(got & 127, want & 127) and np.array_equal(got[:-1], want[:-1])


def test_rounding_by_chance_is_even():
    g = np.random.default_rng(1)
    x = (g.normal(size=256) * 10.0 ** g.uniform(-5, 0, 256)).astype(np.float32)
    total = np.zeros(256)
    n = 4000
    for s in range(n):
        u, _ = ox.chances(7, s, 256)
        codes, scales = ox.round_codes(x, u)
        total += ox.decode(codes) * float(scales[0])
    # a code's step is at most 2^-3 of the value, or 2^-9 of the scale: the mean of n two-valued draws is within
    # 5 / (2 sqrt n) steps of the value (5 standard deviations)
    step = np.maximum(np.abs(x) / 8, float(scales[0]) * 2.0 ** -9)
    assert np.all(np.abs(total / n - x) <= 5 / (2 * np.sqrt(n)) * step)


def test_moments_move_in_8_bits():
    """Nearest codes would leave v at its first value for ever: 0.1 % a step."""
    rng = np.random.default_rng(2)
    f = np.float32
    m = np.zeros(256, f)
    r = np.zeros(256, f)
    g = np.full(256, 1.0) * rng.choice([-1, 1], 256)
    for s in range(1, 1500):
        size = 1.0 if s < 300 else 0.25
        _, _, _, m32, root = ox.adamw(0 * g, size * g, m, (r * r).astype(f), 1e-3, 0.9, 0.999, 1e-8, 0.0, s)
        um, ur = ox.chances(0, s, 256)
        (mc, ms), (rc, rs) = ox.round_codes(m32, um), ox.round_codes(root, ur, floor=True)
        m, r = (ox.decode(mc) * ms[0]).astype(f), (ox.decode(rc) * rs[0]).astype(f)
    exact = np.sqrt(0.999 ** 1200 * (1 - 0.999 ** 299) + 0.0625 * (1 - 0.999 ** 1200))
    # a root's walk: a step of up to 1/8 up or down with the chance of its place gives, over the memory of 2000 steps
    # of the root, a deviation of about a quarter; the mean of 256 is within 5 / 16 of that
    assert abs(r.mean() / exact - 1) < 5 / 16 * 0.25 + 0.05
