"""The forms that only large calls take: gradient lists above 2^26 elements,
read and written past the caches, in every pair of types and in place; sketches
of experts above 2^23 elements in all, whose finished ones are written past the
caches. And calls with a workspace from the caller, which allocate nothing.

Tolerances as for the small calls: the norm 2^-23, a scaled gradient 2^-22 in
fp32 and 2^-8 + 2^-21 in bf16, sketches 1e-5 of their norm and per entry the
products' bound."""
import math

import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from oracle import experts as ox
from rank_gradient_sketching_sketch_amd import binding as B
from gpu_util import device, say, to_f64

pytestmark = pytest.mark.gpu

BIG = (1 << 26) + 12345
TOL = {torch.float32: 2.0 ** -22, torch.bfloat16: 2.0 ** -8 + 2.0 ** -21}


def _gradients(dev, dt, seed):
    """A large tensor off its 16-byte boundary, a short one of the other type, one with gaps between its rows."""
    g = torch.Generator(device=dev).manual_seed(seed)
    other = torch.bfloat16 if dt == torch.float32 else torch.float32
    return [(torch.randn(BIG + 1, generator=g, device=dev) * 1e-2).to(dt)[1:],
            torch.randn(3001, generator=g, device=dev).to(other),
            torch.randn(700, 1016, generator=g, device=dev).to(dt)[:, :1000]]


def _off(got, was, coef):
    """Largest error of got against coef was, in units of the tolerance, a part at a time."""
    worst = 0.0
    got, was = (got.reshape(-1), was.reshape(-1)) if got.is_contiguous() and was.is_contiguous() else (got, was)
    for a, b in zip(got.split(1 << 24), was.split(1 << 24)):
        ref = coef * b.double()
        worst = max(worst, float(((a.double() - ref).abs() / (TOL[got.dtype] * ref.abs() + 2.0 ** -133)).max()))
    return worst


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("to", ["in place", torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ratio", [0.5, 3.0])
def test_clip_past_the_caches(dt, to, ratio):
    dev = device()
    say("large clip", dt, to, ratio)
    grads = _gradients(dev, dt, 3)
    norm_r = math.sqrt(sum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in grads))
    max_norm = float(np.float32(norm_r / ratio))
    coef_r = max_norm / norm_r if norm_r > max_norm else 1.0
    was = [t.clone() for t in grads]
    norm, coef = torch.zeros(1, device=dev), torch.zeros(1, device=dev)
    glist = L.GradList(grads)
    L.logra_grad_norm(glist, norm)
    assert abs(norm.item() - norm_r) <= 2.0 ** -23 * norm_r
    if to == "in place":
        L.logra_grad_clip(glist, max_norm, norm, coef)
        got = grads
    else:
        got = [torch.full(t.shape, 7.0, dtype=to, device=dev) for t in grads]
        L.logra_grad_clip(glist, max_norm, norm, coef, out=L.GradList(got))
        for t, w in zip(grads, was):
            assert torch.equal(t, w)
    assert abs(norm.item() - norm_r) <= 2.0 ** -23 * norm_r and abs(coef.item() - coef_r) <= 2.0 ** -23 * coef_r
    for t, w in zip(got, was):
        assert _off(t, w, coef_r) <= 1.0


@pytest.mark.parametrize("T,K,E,d,r,popular", [(2100, 2, 40, 1024, 256, 7), (90, 2, 600, 256, 64, None)])
def test_sketches_past_the_caches(T, K, E, d, r, popular):
    """Experts whose rows are split over items, experts of one item and
    experts without rows beside each other."""
    dev = device()
    assert E * d * r > 8 << 20
    say("large expert sketches", T, K, E, d, r, popular)
    g = np.random.default_rng(T)
    k = 136
    ids = g.integers(0, E, (T, K))
    if popular is not None:
        ids = np.where(g.random((T, K)) < 0.7, popular, ids % (E - 3))
    offsets, order, _ = (torch.from_numpy(x).to(dev) for x in ox.expert_sort(ids, E))
    tg = torch.Generator().manual_seed(T)
    X = torch.randn(T, k, generator=tg).to(torch.bfloat16).to(dev)
    dY = (torch.randn(T * K, d, generator=tg) * 1e-3).to(torch.bfloat16).to(dev)
    m = L.MatrixDesc(d, k, r, seed=5, step=2, matrix_id=40)
    S = torch.full((E, d, r), float("nan"), device=dev)
    L.logra_sketch_experts(m, offsets, X, dY, S, False, order=order, topk=K)
    o = offsets.cpu().numpy()
    counts = np.diff(o)
    assert (counts == 0).any() and (popular is None or counts[popular] > 2000)
    ref, mag_p, mag_x = ox.sketch_experts(to_f64(X), to_f64(dY), o, d, k, r, 5, 2, 40, 1, order=order.cpu().numpy(), topk=K)
    bound = (2.0 ** -24 + (3 * counts.max() + 16) * 2.0 ** -23) * mag_p + (k + 16) * 2.0 ** -23 * (1 + 2.0 ** -8) * mag_x
    for times in (1, 2):
        got = to_f64(S)
        assert np.all(np.abs(got - times * ref) <= times * bound + 1e-30)
        assert np.linalg.norm(got - times * ref) <= 1e-5 * times * np.linalg.norm(ref)
        assert not got[counts == 0].any()
        L.logra_sketch_experts(m, offsets, X, dY, S, True, order=order, topk=K)


def test_calls_with_a_workspace_allocate_nothing():
    dev = device()
    T, K, E, h, d, r = 5000, 2, 16, 96, 64, 128
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(-1, E, (T, K), generator=g).to(dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    order = torch.empty(T * K, dtype=torch.int32, device=dev)
    slots = torch.empty(T, K, dtype=torch.int32, device=dev)
    w, dw = torch.rand(T, K, generator=g).to(dev), torch.empty(T, K, device=dev)
    X, Y = torch.randn(T, h, generator=g).to(dev).bfloat16(), torch.empty(T, h, device=dev).bfloat16()
    Xs, dXs = torch.zeros(T * K, h, device=dev).bfloat16(), torch.zeros(T * K, h, device=dev).bfloat16()
    dYs = torch.randn(T * K, d, generator=g).to(dev).bfloat16()
    S, out = torch.empty(E, d, r, device=dev), torch.empty(E, d, r, device=dev)
    m = L.MatrixDesc(d, h, r)
    lists = L.GradList([S]), L.GradList([out])
    norm, coef = torch.empty(1, device=dev), torch.empty(1, device=dev)

    def ws(n):
        assert n > 0
        return torch.empty(n, dtype=torch.uint8, device=dev)

    ws_sort = ws(L.logra_expert_sort_workspace_bytes(T, K, E))
    ws_sketch = ws(L.logra_sketch_experts_workspace_bytes(m, E, T * K, B.LOGRA_BF16))
    ws_clip = ws(L.logra_grad_workspace_bytes(lists[0]))

    def calls(**kw):
        L.logra_expert_sort(ids, E, offsets, order, slots, ws=ws_sort, **kw)
        L.logra_expert_gather(X, slots, Xs, weights=w, **kw)
        L.logra_expert_combine(Xs, slots, Y, weights=w, **kw)
        L.logra_expert_combine_backward(X, Xs, slots, w, dXs, dw, **kw)
        L.logra_sketch_experts(m, offsets, X, dYs, S, False, order=order, topk=K, ws=ws_sketch, **kw)
        L.logra_sketch_experts(m, offsets, Xs, dYs, S, True, ws=ws_sketch, **kw)
        L.logra_grad_norm(lists[0], norm, ws=ws_clip, **kw)
        L.logra_grad_clip(lists[0], 1.0, norm, coef, out=lists[1], ws=ws_clip, **kw)
        L.logra_grad_clip(lists[0], 1.0, norm, coef, ws=ws_clip, **kw)

    side = torch.cuda.Stream(device=dev)
    calls()
    torch.cuda.synchronize()
    calls(stream=side)
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats(dev)["allocation.all.allocated"]
    for _ in range(3):
        calls()
        torch.cuda.synchronize()
        calls(stream=side)
        torch.cuda.synchronize()
    assert torch.cuda.memory_stats(dev)["allocation.all.allocated"] == before
