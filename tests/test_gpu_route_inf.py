"""Logits of +inf where keys are formed (a bias, or sums of a group's two best):
a softmax has no values there, so experts are chosen as where logits are
compared, and the weights are NaN, which shows, instead of the token's rows
being dropped like a padding token's. A sigmoid of +inf is 1."""
import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from oracle import layers as ox
from gpu_util import device

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
E = 40


def _route(x, K, score, dev, bias=None, **kw):
    ids = torch.full((x.shape[0], K), -77, dtype=torch.int32, device=dev)
    w = torch.zeros(x.shape[0], K, device=dev)
    L.logra_route(x.to(dev), ids, w, bias=None if bias is None else bias.to(dev), score=score, **kw)
    return ids.cpu().numpy(), w.cpu().double().numpy()


def _logits():
    x = 2 * torch.randn(9, E, generator=torch.Generator().manual_seed(6))
    x[1, 17] = INF
    x[2, 3] = x[2, 31] = INF
    x[3, :] = INF
    x[4, 5], x[4, 6] = INF, NAN
    x[5, 1:] = -INF
    x[5, 0] = INF
    x[6, 9], x[6, 10:] = INF, -INF
    x[7] = -INF
    return x


GROUPED = dict(groups=8, topk_groups=3, group_best=2)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("biased,kw", [(True, {}), (True, GROUPED), (False, GROUPED), (True, dict(GROUPED, group_best=1))])
def test_inf(biased, kw, renorm, dt):
    dev = device()
    x = _logits().to(dt)
    bias = 0.3 * torch.randn(E, generator=torch.Generator().manual_seed(7)) if biased else None
    b = None if bias is None else bias.double().numpy()
    xr = x.double().numpy()
    ids, w = _route(x, 6, ox.SOFTMAX, dev, bias, renormalize=renorm, **kw)
    ref_ids, ref_w = ox.route(xr, 6, ox.SOFTMAX, b, renormalize=renorm, **kw)
    assert np.array_equal(ids, ref_ids) and np.array_equal(np.isnan(w), np.isnan(ref_w))
    rows = np.array([1, 2, 3, 4, 5, 6])
    assert np.all(xr[rows, ids[rows, 0]] == INF)                # the first choice is one of those with +inf
    assert np.array_equal(np.isnan(w[rows]), ids[rows] >= 0)    # and what was chosen has no weight
    assert np.all(ids[7] == -1) and not w[7].any()
    ids, w = _route(x, 6, ox.SIGMOID, dev, bias, renormalize=renorm, **kw)
    ref_ids, ref_w = ox.route(xr, 6, ox.SIGMOID, b, renormalize=renorm, **kw)
    assert np.array_equal(ids, ref_ids) and np.array_equal(np.isnan(w), np.isnan(ref_w))
    ok = ~np.isnan(w)
    # finite logits are below 12; a sigmoid of +inf has no rounding
    assert np.all(np.abs(w - ref_w)[ok] <= (2 * 24 + 48) * 2.0 ** -24 * np.abs(ref_w)[ok])


def test_inf_beside_a_bias_that_has_none():
    """An expert without a key is not chosen, whatever its logit; without any other the token has no expert."""
    dev = device()
    x = torch.zeros(2, E)
    x[0, 4] = x[0, 8] = x[1, 4] = INF
    x[1, 5:] = x[1, :4] = -INF
    bias = torch.zeros(E)
    bias[4] = -INF
    for nothing in (-INF, NAN):
        bias[4] = nothing
        ids, w = _route(x, 2, ox.SOFTMAX, dev, bias)
        assert ids.tolist() == [[8, 0], [-1, -1]] and np.isnan(w[0]).all() and not w[1].any()
