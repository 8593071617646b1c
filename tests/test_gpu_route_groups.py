"""Groups of experts whose two best keys nearly cancel: biases of both signs make
keys whose rounding in fp32 is far above that of their sum, and the groups that
stay must be those of keys in fp64. Ids: equal to the fp64 form's. Weights: the
bias is not part of them, (2 D + 48) 2^-24 of the weight as for any routing,
with D twice the largest logit."""
import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from oracle import layers as ox
from gpu_util import device, say

pytestmark = pytest.mark.gpu


def _check(x, K, score, bias, **kw):
    dev = device()
    T = x.shape[0]
    ids = torch.full((T, K), -77, dtype=torch.int32, device=dev)
    w = torch.full((T, K), float("nan"), device=dev)
    L.logra_route(torch.from_numpy(x).to(dev), ids, w, bias=torch.from_numpy(bias).to(dev), score=score, **kw)
    ref_ids, ref_w = ox.route(x, K, score, bias, **kw)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    D = 2 * float(np.abs(x).max())
    assert np.all(np.abs(w.cpu().double().numpy() - ref_w) <= (2 * D + 48) * 2.0 ** -24 * np.abs(ref_w))


def test_one_token():
    x = np.array([[0.17640908, 0.46769133, -0.62792438, 1.45550537]], np.float32)
    bias = np.array([16, -16, 16, -16], np.float32)
    _check(x, 1, ox.SIGMOID, bias, groups=2, topk_groups=1, group_best=2)
    assert ox.route(x, 1, ox.SIGMOID, bias, groups=2, topk_groups=1, group_best=2)[0][0, 0] == 2


def _biases(g, groups, size, B):
    """B for one expert of every group, -B for the others."""
    b = np.full((groups, size), -B)
    b[np.arange(groups), g.integers(0, size, groups)] = B
    return b


@pytest.mark.parametrize("B", [0.5, 2.0, 8.0, 64.0, 1e4])
@pytest.mark.parametrize("groups,size,kept", [(2, 2, 1), (3, 20, 2), (8, 32, 4), (16, 10, 3), (64, 16, 9)])
def test_sigmoid(groups, size, kept, B):
    """Sums of the two best keys within some roundings of B of each other."""
    say("sigmoid", groups, size, kept, B)
    g = np.random.default_rng(groups + size)
    T = 500
    b = _biases(g, groups, size, B)
    s = 0.1 + 0.5 * g.random((T, groups, size))
    second = np.where(b > 0, 0.0, s).max(2)                     # the best of those with -B
    top = 1.1 - second + max(B, 1.0) * 2.0 ** -22 * g.uniform(-1, 1, second.shape)
    s = np.clip(np.where(b > 0, top[:, :, None], s), 0.02, 0.98)
    x = np.log(s / (1 - s)).reshape(T, -1).astype(np.float32)
    bias = b.reshape(-1).astype(np.float32)
    for best in (2, 1):
        _check(x, min(6, kept * size), ox.SIGMOID, bias, groups=groups, topk_groups=kept, group_best=best)


@pytest.mark.parametrize("B", [0.5, 2.0, 8.0, 64.0, 1e4])
@pytest.mark.parametrize("groups,size,kept,spread", [(8, 128, 4, 1e-3), (64, 16, 9, 1e-2), (32, 2, 7, 1.0), (8, 32, 4, 2.0)])
def test_softmax(groups, size, kept, spread, B):
    """Many experts of nearly the same score, whose keys are rounded at the bias's size."""
    say("softmax", groups, size, kept, B)
    g = np.random.default_rng(groups + size)
    x = (spread * g.standard_normal((500, groups * size))).astype(np.float32)
    bias = _biases(g, groups, size, B).reshape(-1).astype(np.float32)
    for best in (2, 1):
        _check(x, min(6, kept * size), ox.SOFTMAX, bias, groups=groups, topk_groups=kept, group_best=best)


def test_one_group_of_large_keys():
    """The groups at the border have small keys and are told apart; a third one's large keys cancel and may be anywhere."""
    g = np.random.default_rng(5)
    T = 2000
    bias = np.array([4096, -4096, 0, 0, 0, 0], np.float32)
    s = 0.3 + 0.2 * g.random((T, 6))
    s[:, 0] = s[:, 2] + s[:, 3] - s[:, 1] + 2.0 ** -11 * g.uniform(-1, 1, T)
    s[:, 4] = s[:, 2] - 1e-4                                    # the third group is just below the second
    s[:, 5] = s[:, 3]
    s = np.clip(s, 0.02, 0.98)
    x = np.log(s / (1 - s)).astype(np.float32)
    _check(x, 2, ox.SIGMOID, bias, groups=3, topk_groups=2, group_best=2)
    _check(x, 2, ox.SIGMOID, bias, groups=3, topk_groups=1, group_best=2)
