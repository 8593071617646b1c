"""Routing and its gradient against the plain fp64 form.

Tolerances. Ids: equal. A weight is a ratio of exponentials of differences of
logits: the difference d is rounded once (2^-24 |d|), the exponential is within
2^-23 of its argument's, a sum of n positive terms adds at most (n + 6) 2^-24
where n is a lane's own terms (16 at most) and 6 are the steps over the wave, a
sigmoid adds its own exponential, sum and quotient, and quotient and scale one
rounding each: (2 D + 48) 2^-24 of the weight with D the largest |d| covers
numerator and denominator. The gradient is products of such weights and sums
over the choices of terms whose magnitudes the oracle adds up: (4 D + 128 + K)
2^-24 of those, then the rounding to bf16 (2^-8)."""
import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from oracle import layers as ox
from gpu_util import device, say

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def _logits(seed, T, E, dt, dev, pad=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    base = (spread * torch.randn(T, E + pad, generator=g)).to(dt).to(dev)
    return base[:, pad // 2:pad // 2 + E] if pad else base


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _run(x, K, score, bias=None, **kw):
    T = x.shape[0]
    ids = torch.full((T, K), -77, dtype=torch.int32, device=x.device)
    w = torch.full((T, K), NAN, device=x.device)
    L.logra_route(x, ids, w, bias=bias, score=score, **kw)
    return ids, w


def _check(x, K, score, bias=None, **kw):
    ids, w = _run(x, K, score, bias, **kw)
    xr = _f64(x)
    ref_ids, ref_w = ox.route(xr, K, score, None if bias is None else _f64(bias), **kw)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    live = np.where(np.isfinite(xr), xr, np.nan)
    D = 0.0 if not np.isfinite(live).any() else 2 * float(np.nanmax(np.abs(live)))
    w = _f64(w)
    assert np.array_equal(np.isnan(w), np.isnan(ref_w))
    ok = ~np.isnan(w)
    assert np.all(np.abs(w - ref_w)[ok] <= (2 * D + 48) * 2.0 ** -24 * np.abs(ref_w)[ok])
    return ids


SHAPES = [(0, 4, 2), (1, 1, 1), (1, 128, 8), (3, 3, 3), (5, 60, 4), (64, 64, 8), (17, 65, 6), (9, 128, 64), (333, 129, 8),
          (100, 256, 8), (7, 500, 1), (6, 1000, 33), (5, 1024, 64), (70001, 16, 2)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [ox.SOFTMAX, ox.SIGMOID])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_route(T, E, K, score, dt):
    dev = device()
    say("route", T, E, K, score, dt)
    x = _logits(T + E, T, E, dt, dev, pad=3 if E % 2 else 0)
    bias = 0.3 * torch.randn(E, generator=torch.Generator().manual_seed(E)).to(dev)
    few = T > 1000
    for b in ((bias,) if few else (None, bias)):
        for renorm in ((True,) if few else (True, False)):
            _check(x, K, score, b, renormalize=renorm, scale=2.5)


# groups, experts, kept, of which the lanes' spans are 32, 16, 8, 4, 2, 1, whole and ragged
GROUPS = [(2, 8, 1), (3, 60, 2), (4, 64, 2), (5, 35, 4), (8, 256, 4), (8, 1024, 1), (9, 1017, 3), (16, 160, 3), (17, 1020, 5),
          (32, 64, 7), (33, 1023, 8), (60, 60, 2), (64, 1024, 9), (4, 64, 4), (1, 40, 1)]


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("groups,E,kept", GROUPS)
def test_route_groups(groups, E, kept, best):
    dev = device()
    say("groups", groups, E, kept, best)
    for dt, score, biased in ((torch.float32, ox.SIGMOID, True), (torch.bfloat16, ox.SOFTMAX, False), (torch.float32, ox.SOFTMAX, True),
                              (torch.float32, ox.SIGMOID, False)):
        x = _logits(E + groups, 50, E, dt, dev)
        x[3, : E // 2] = -INF                                   # groups with one expert to choose, or none
        x[4, 1:] = -INF
        bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E)).to(dev) if biased else None
        for K in (1, min(E, 6), min(E, 64)):
            _check(x, K, score, bias, groups=groups, topk_groups=kept, group_best=best, renormalize=True)


@pytest.mark.parametrize("alike", [2, 3, 9, 15, 16, 17, 40, 256])
@pytest.mark.parametrize("K", [1, 7, 8, 60, 64])
def test_route_keys_that_fp32_cannot_tell(K, alike):
    """Some experts' keys within fp32 rounding of each other, above or below others; some equal; ids stay those of fp64 keys."""
    dev = device()
    E, T = 256, 48
    g = np.random.default_rng(K * 1000 + alike)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    x = (g.standard_normal((T, E)) - 2.0).astype(np.float32)
    for t in range(T):
        pick = g.choice(E, alike, replace=False)
        c = 0.5 + 0.1 * g.random()
        s = c - bias[pick].astype(np.float64)
        x[t, pick] = np.log(s / (1 - s)).astype(np.float32)
        x[t, pick[:alike // 3]] = np.nextafter(x[t, pick[:alike // 3]], np.float32(9))
        rest = np.setdiff1d(np.arange(E), pick)
        up = g.choice(rest, min(len(rest), t % 12), replace=False)
        x[t, up] += 5.0
    x[T - 2:] = x[T - 2:, :1]                                   # all logits equal
    y = x.copy()
    y[:, 1::2] = y[:, ::2]                                      # and pairs of equal keys
    twice = bias.copy()
    twice[1::2] = twice[::2]
    for logits, b in ((x, bias), (y, twice), (y, np.zeros_like(bias))):
        for kw in (dict(), dict(groups=8, topk_groups=4, group_best=2)):
            _check(torch.from_numpy(logits).to(dev), K, ox.SIGMOID, torch.from_numpy(b).to(dev), renormalize=True, **kw)
    _check(torch.from_numpy(x).to(dev), K, ox.SOFTMAX, torch.from_numpy(bias).to(dev), renormalize=True)


@pytest.mark.parametrize("score", [ox.SOFTMAX, ox.SIGMOID])
def test_route_edges(score):
    dev = device()
    E = 40
    x = _logits(1, 24, E, torch.float32, dev)
    x[0] = -INF                          # a padding token
    x[1] = 0.0                           # all equal: the lowest indexes
    x[2, ::2], x[2, 1::2] = 0.0, -0.0    # both zeros are one value
    x[3, 5], x[3, 9] = NAN, 3e38
    x[4] = NAN
    x[5, 2:] = -INF                      # fewer than are asked for
    x[6] = torch.finfo(torch.float32).min                       # a mask of the type's lowest value
    x[7, 1:] = torch.finfo(torch.float32).min
    x[8] = -80.0 - torch.arange(E, device=dev) / 8.0            # sigmoids that vanish in fp32
    x[9] = 30.0 + torch.arange(E, device=dev) / 8.0             # ... that are 1 in fp32
    x[10, 7] = x[10, 30] = x[10].max() + 1                      # a tie at the top
    x[11] = x[11] * 1e-30
    bias = torch.zeros(E, device=dev)
    for renorm in (True, False):
        ids, w = _run(x, 8, score, renormalize=renorm)
        ref_ids, ref_w = ox.route(_f64(x), 8, score, renormalize=renorm)
        assert np.array_equal(ids.cpu().numpy(), ref_ids)
        got = _f64(w)
        assert np.array_equal(np.isnan(got), np.isnan(ref_w))
        ok = ~np.isnan(got)
        # rows 8 and 9 spread over 5 logits, row 3 over 3e38: there a weight is 1 or 0. D = 12 elsewhere. A weight
        # below 2^-126 keeps its last bit alone.
        assert np.all(np.abs(got - ref_w)[ok] <= (2 * 12 + 48) * 2.0 ** -24 * np.abs(ref_w)[ok] + 2.0 ** -126)
    bias[3], bias[4], bias[5] = -INF, NAN, 100.0
    ids, _ = _run(x, 8, score, bias=bias)
    assert np.array_equal(ids.cpu().numpy(), ox.route(_f64(x), 8, score, _f64(bias))[0])
    assert not ((ids == 3) | (ids == 4)).any()
    # +inf: taken first where logits are compared; its sigmoid is 1, its softmax has no value
    x = torch.zeros(1, E, device=dev)
    x[0, 17] = INF
    ids, w = _run(x, 2, score, renormalize=False)
    assert ids.tolist() == [[17, 0]] and (torch.isnan(w).all() if score == ox.SOFTMAX else w.tolist() == [[1.0, 0.5]])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [ox.SOFTMAX, ox.SIGMOID])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_route_backward(T, E, K, score, dt):
    dev = device()
    say("route backward", T, E, K, score, dt)
    x = _logits(T + 2 * E, T, E, dt, dev, pad=5 if E % 2 else 0)
    if T > 2:
        x[2] = -INF
    ids, _ = _run(x, K, score)
    g = torch.Generator().manual_seed(T + K)
    if T > 4:
        ids[1, 0] = -1                              # dropped after the choice
        ids[3, -1] = E + 3                          # not there
        ids[4, -1] = ids[4, 0]                      # the same expert twice
    dw = torch.randn(T, K, generator=g).to(dev)
    dx = torch.full_like(x, NAN) if x.is_contiguous() else torch.full((T, E + 7), NAN, dtype=dt, device=dev)[:, 2:2 + E]
    half = 2.0 ** -8 if dt == torch.bfloat16 else 0.0
    for renorm in (True, False):
        dx.fill_(NAN)
        L.logra_route_backward(x, ids, dw, dx, score=score, renormalize=renorm, scale=1.5)
        ref, mag = ox.route_backward(_f64(x), ids.cpu().numpy(), _f64(dw), score, renorm, 1.5)
        err = np.abs(_f64(dx) - ref)
        D = 4 * 6.0                                 # logits of a deviation of 2 stay below 12
        assert np.all(err <= half * np.abs(ref) + (1 + half) * (4 * D + 128 + K) * 2.0 ** -24 * mag + 2.0 ** -126)


def test_route_backward_in_place_and_differences():
    dev = device()
    x = _logits(8, 31, 48, torch.float32, dev)
    ids, w = _run(x, 5, ox.SIGMOID, scale=2.0)
    dw = torch.randn(31, 5, generator=torch.Generator().manual_seed(2)).to(dev)
    dx = torch.empty_like(x)
    L.logra_route_backward(x, ids, dw, dx, score=ox.SIGMOID, scale=2.0)
    # against differences of the fp64 form: h^2 / 6 of a third derivative of order one, and 2^-53 / h
    h, xr, i, d = 1e-5, _f64(x), ids.cpu().numpy(), _f64(dw)
    for e in range(48):
        up, down = xr.copy(), xr.copy()
        up[:, e] += h
        down[:, e] -= h
        slope = ((ox.route_weights(up, i, 1, True, 2.0) - ox.route_weights(down, i, 1, True, 2.0)) * d).sum(1) / (2 * h)
        assert np.all(np.abs(slope - _f64(dx)[:, e]) < 1e-5)
    same = x.clone()
    L.logra_route_backward(same, ids, dw, same, score=ox.SIGMOID, scale=2.0)
    assert torch.equal(same, dx)


def test_route_streams_and_graph():
    dev = device()
    side = torch.cuda.Stream()
    x = _logits(4, 700, 128, torch.float32, dev)
    ids, w = _run(x, 8, ox.SOFTMAX)
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    side.wait_stream(torch.cuda.current_stream())
    L.logra_route(x, ids2, w2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    static, dx = x.clone(), torch.empty_like(x)
    dw = torch.randn(700, 8, generator=torch.Generator().manual_seed(3)).to(dev)
    L.logra_route(static, ids2, w2)
    L.logra_route_backward(static, ids2, dw, dx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.logra_route(static, ids2, w2)
        L.logra_route_backward(static, ids2, dw, dx)
    for seed in (11, 12, 13):
        static.copy_(_logits(seed, 700, 128, torch.float32, dev))
        graph.replay()
        torch.cuda.synchronize()
        want = _run(static, 8, ox.SOFTMAX)
        dx3 = torch.empty_like(dx)
        L.logra_route_backward(static, want[0], dw, dx3)
        assert torch.equal(ids2, want[0]) and torch.equal(w2, want[1]) and torch.equal(dx, dx3)
    with pytest.raises(L.LograError):
        L.logra_route(x, ids.cpu(), w)
