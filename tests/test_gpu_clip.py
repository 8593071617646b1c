"""Global gradient norm and clipping against the fp64 oracle.

Tolerances. The squares and sums are fp64 (relative error below n 2^-53), so
the stored norm and factor are each one fp32 rounding, 2^-24, off (2^-23 with
the fp64 sum allowed for); a scaled gradient adds the product's rounding
(2^-24) and, in bf16, its own (2^-8)."""
import math

import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from oracle import experts as ox
from gpu_util import device, say

pytestmark = pytest.mark.gpu

F32_OUT = 2.0 ** -22
BF16_OUT = 2.0 ** -8 + 2.0 ** -21


def _scalars(dev):
    return torch.full((1,), float("nan"), device=dev), torch.full((1,), float("nan"), device=dev)


def _check(got, ref, dtype):
    got, ref = got.detach().cpu().double().numpy(), np.asarray(ref)
    tol = BF16_OUT if dtype == torch.bfloat16 else F32_OUT
    tiny = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149
    assert np.all(np.abs(got - ref) <= tol * np.abs(ref) + tiny)


def _mixed(dev, seed, shapes, odd=0):
    """Tensors of alternating type laid out one after another in one buffer
    per type, `odd` elements in, so most start off a 16-byte boundary."""
    g = torch.Generator().manual_seed(seed)
    sizes = {torch.float32: odd, torch.bfloat16: odd}
    for i, s in enumerate(shapes):
        sizes[torch.bfloat16 if i % 2 else torch.float32] += math.prod(s)
    flat = {k: (torch.randn(n + 8, generator=g) * 1e-2).to(k).to(dev) for k, n in sizes.items()}
    at = {torch.float32: odd, torch.bfloat16: odd}
    out = []
    for i, s in enumerate(shapes):
        k = torch.bfloat16 if i % 2 else torch.float32
        out.append(flat[k][at[k]:at[k] + math.prod(s)].view(s))
        at[k] += math.prod(s)
    return out, flat


SHAPES = [
    [(1,)],
    [(3,), (5,)],
    [(256, 32), (1536,), (7, 11), (1,), (0,), (300, 3)],
    [(8192,), (8193,), (8191,), (2, 8200), (16385,)],
    [(1000, 256), (1000, 255), (17,), (40000, 1), (3, 50001)],
]


@pytest.mark.parametrize("odd", [0, 1, 3])
@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("ratio", [0.5, 3.0])
def test_clip_matches_oracle(case, odd, ratio):
    dev = device()
    say("clip", SHAPES[case], odd, ratio)
    grads, flat = _mixed(dev, 10 * case + odd, SHAPES[case], odd)
    before = {k: v.clone() for k, v in flat.items()}
    ref = [g.cpu().double().numpy() for g in grads]
    norm0, _, _ = ox.clip(ref, math.inf)
    max_norm = float(np.float32(norm0 / ratio))
    norm_r, coef_r, out_r = ox.clip(ref, max_norm)
    glist = L.GradList(grads)
    assert glist.elements == sum(g.numel() for g in grads)
    norm, coef = _scalars(dev)
    L.logra_grad_norm(glist, norm)
    assert abs(norm.item() - norm_r) <= 2.0 ** -23 * norm_r
    # into other tensors of the other type: the gradients stay
    others = [torch.full_like(g, 9.0, dtype=torch.float32 if g.dtype == torch.bfloat16 else torch.bfloat16)
              for g in grads]
    norm, coef = _scalars(dev)
    L.logra_grad_clip(glist, max_norm, norm, coef, out=L.GradList(others))
    for k in flat:
        assert torch.equal(flat[k], before[k])
    for o, r in zip(others, out_r):
        _check(o, r, o.dtype)
    # in place; nothing around the tensors changes
    norm, coef = _scalars(dev)
    L.logra_grad_clip(glist, max_norm, norm, coef)
    assert abs(norm.item() - norm_r) <= 2.0 ** -23 * norm_r
    assert abs(coef.item() - coef_r) <= 2.0 ** -23 * coef_r
    for g, r in zip(grads, out_r):
        _check(g, r, g.dtype)
    if ratio < 1:
        assert coef.item() == 1.0
        for k in flat:
            assert torch.equal(flat[k], before[k])
    for k in flat:
        used = odd + sum(g.numel() for g in grads if g.dtype == k)
        assert torch.equal(flat[k][:odd], before[k][:odd]) and torch.equal(flat[k][used:], before[k][used:])


def test_strided_tensors_and_copies_between_layouts():
    dev = device()
    g = torch.Generator().manual_seed(4)
    shapes = [(37, 20, 32), (5, 9001, 9100), (300, 1, 5), (64, 256, 512), (3, 7, 7)]
    for dt in (torch.float32, torch.bfloat16):
        bases = [torch.randn(r, ld, generator=g).to(dt).to(dev) for r, c, ld in shapes]
        views = [b[:, ld - c:] for b, (r, c, ld) in zip(bases, shapes)]
        keep = [b.clone() for b in bases]
        dense = [torch.zeros(r, c, dtype=dt, device=dev) for r, c, _ in shapes]
        norm_r, coef_r, out_r = ox.clip([v.cpu().double().numpy() for v in views], 2.5)
        norm, coef = _scalars(dev)
        L.logra_grad_clip(L.GradList(views), 2.5, norm, coef, out=L.GradList(dense))
        for d, r in zip(dense, out_r):
            _check(d, r, dt)
        # the other way round, and in place
        L.logra_grad_clip(L.GradList(dense), math.inf, norm, coef, out=L.GradList(views))
        for v, d, b, k, (r, c, ld) in zip(views, dense, bases, keep, shapes):
            assert torch.equal(v, d)
            assert torch.equal(b[:, :ld - c], k[:, :ld - c])
        L.logra_grad_clip(L.GradList(views), 1.0, norm, coef)
        n2, c2, o2 = ox.clip([d.cpu().double().numpy() for d in dense], 1.0)
        assert abs(norm.item() - n2) <= 2.0 ** -23 * n2
        for v, r, b, k, (rr, c, ld) in zip(views, o2, bases, keep, shapes):
            _check(v, r, dt)
            assert torch.equal(b[:, :ld - c], k[:, :ld - c])


def test_many_tensors_and_empty_lists():
    dev = device()
    g = torch.Generator().manual_seed(1)
    sizes = torch.randint(0, 400, (5000,), generator=g).tolist()
    flat = torch.randn(sum(sizes), generator=g).to(dev)
    grads = list(torch.split(flat, sizes))
    norm, coef = _scalars(dev)
    ref = flat.double().norm().item()
    L.logra_grad_clip(L.GradList(grads), 1.0, norm, coef)
    assert abs(norm.item() - ref) <= 2.0 ** -23 * ref
    assert abs(flat.double().norm().item() - 1.0) <= 2.0 ** -22
    for empty in (L.GradList([], device=dev), L.GradList([torch.empty(0, 5, device=dev)])):
        norm, coef = _scalars(dev)
        L.logra_grad_clip(empty, 1.0, norm, coef)
        assert norm.item() == 0.0 and coef.item() == 1.0
        L.logra_grad_norm(empty, norm)
        assert norm.item() == 0.0


def test_extreme_values():
    dev = device()
    norm, coef = _scalars(dev)
    for v in (1e30, 3e38, 1e-30, 1e-42):       # squares far outside the fp32 range
        x = torch.full((1000,), v, device=dev)
        exact = float(x[0].double()) * math.sqrt(1000)
        L.logra_grad_norm(L.GradList([x]), norm)
        want = np.float32(exact) if exact < 3.4e38 else np.float32(np.inf)
        assert np.isinf(want) == math.isinf(norm.item())
        if np.isfinite(want):
            assert abs(norm.item() - exact) <= 2.0 ** -23 * exact + 2.0 ** -149
    x = torch.full((1000,), 3e38, device=dev)      # the norm above the fp32 range still clips right
    L.logra_grad_clip(L.GradList([x]), 1.0, norm, coef)
    assert abs(x.double().norm().item() - 1.0) < 2.0 ** -9     # the factor is subnormal: 2^-149 of 1e-40
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.randn(5000, generator=torch.Generator().manual_seed(0)).to(dev)
        x[4321] = bad
        keep = x.clone()
        L.logra_grad_clip(L.GradList([x]), 1e-3, norm, coef)
        assert not math.isfinite(norm.item()) and coef.item() == 1.0
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(keep))
    x = torch.randn(100, generator=torch.Generator().manual_seed(0)).to(dev)
    L.logra_grad_clip(L.GradList([x]), 0.0, norm, coef)
    assert coef.item() == 0.0 and not x.any()


def test_one_tensor_past_32_bit_offsets():
    dev = device()
    n = (1 << 31) + 40001
    x = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    where = [0, 12345, (1 << 30) + 7, (1 << 31) - 1, 1 << 31, n - 1]
    for i, p in enumerate(where):
        x[p] = 2.0 ** i
    norm, coef = _scalars(dev)
    exact = math.sqrt(sum(4.0 ** i for i in range(len(where))))
    L.logra_grad_clip(L.GradList([x]), float(np.float32(exact / 2)), norm, coef)
    assert abs(norm.item() - exact) <= 2.0 ** -23 * exact
    for i, p in enumerate(where):
        assert abs(float(x[p]) - 2.0 ** (i - 1)) <= BF16_OUT * 2.0 ** (i - 1)
    assert int(torch.count_nonzero(x)) == len(where)


def test_repeats_graphs_and_streams():
    dev = device()
    grads, flat = _mixed(dev, 77, [(513, 256), (1536,), (300, 64), (9,)], 1)
    keep = {k: v.clone() for k, v in flat.items()}
    glist = L.GradList(grads)
    norm, coef = _scalars(dev)
    ws = torch.empty(L.logra_grad_workspace_bytes(glist), dtype=torch.uint8, device=dev)

    def reset():
        for k in flat:
            flat[k].copy_(keep[k])

    L.logra_grad_clip(glist, 0.5, norm, coef, ws=ws)
    torch.cuda.synchronize()
    ref = (norm.clone(), coef.clone(), {k: v.clone() for k, v in flat.items()})

    def same():
        torch.cuda.synchronize()
        assert torch.equal(norm, ref[0]) and torch.equal(coef, ref[1])
        for k in flat:
            assert torch.equal(flat[k], ref[2][k])

    for _ in range(3):
        reset()
        L.logra_grad_clip(glist, 0.5, norm, coef, ws=ws)
        same()
    side = torch.cuda.Stream()
    for _ in range(3):                 # a stream of its own, workspace from the binding
        reset()
        side.wait_stream(torch.cuda.current_stream())
        L.logra_grad_clip(glist, 0.5, norm, coef, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        junk = torch.full((1 << 16,), 255, dtype=torch.uint8, device=dev)
        same()
        del junk
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.logra_grad_clip(glist, 0.5, norm, coef, ws=ws)
    for _ in range(3):
        reset()
        L.logra_grad_clip(glist, 0.5, norm, coef)
        reset()
        norm.zero_(), coef.zero_()
        torch.cuda.synchronize()
        graph.replay()
        same()
