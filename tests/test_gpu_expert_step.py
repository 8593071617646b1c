"""The expert-layer calls, clipping and the optimizer step used together, as a
training program uses them: tokens sorted by expert and gathered, the experts'
products, the weighted combination, its gradient, the sketch over experts and
of a dense projection beside it, clipping by the global norm, both apply
passes. Every stage is checked against an fp64 computation of the whole chain
that starts from the same inputs (the products in between, which the library
does not do, are torch's on the GPU).

Tolerance: the bf16 path's 2e-2 per row (gpu_util.BF16_TOL): every stage rounds
its result to bf16 once (2^-8) and the sketch of the dense projection rounds
its projection; the apply passes round S (2^-8)."""
import numpy as np
import pytest
import torch

import oracle
import rank_gradient_sketching_sketch_amd as L
from oracle import experts as ox
from rank_gradient_sketching_sketch_amd import binding as B
from rank_gradient_sketching_sketch_amd.step import ExpertGroup, Matrix, Step
from gpu_util import BF16_TOL, device, f32, rel_err, rownorm_err, say, to_f64, w_update_err

pytestmark = pytest.mark.gpu

T, K, E, D, H, R = 200, 2, 6, 64, 96, 64      # tokens, choices, experts, rows and columns of W, rank
MBS, BETA2, EPS, LR = 2, 0.99, 1e-8, 1e-3


def _layer(dev, mb):
    """One microbatch's forward and backward pass through the layer, on the
    GPU, and the same in fp64."""
    g = torch.Generator().manual_seed(100 + mb)
    logits = torch.randn(T, E, generator=g)
    top, ids = torch.topk(logits, K, dim=1)
    ids[-7:] = -1                                             # padding tokens
    w = torch.softmax(top, 1)
    X = torch.randn(T, H, generator=g).to(torch.bfloat16)
    dY = (torch.randn(T, D, generator=g) * 1e-2).to(torch.bfloat16)
    return ids, w, X, dY


@pytest.mark.parametrize("max_norm", [1e-3, 1e6])
def test_layer_and_step(max_norm):
    dev = device()
    g = torch.Generator().manual_seed(9)
    W = torch.randn(E, D, H, generator=g) * 0.1
    Wd = torch.randn(40, H, generator=g) * 0.1                # a dense projection that reads the same X
    gains = torch.randn(H + 1, generator=g) * 1e-2            # a dense gradient beside the sketches
    say("expert step", max_norm)
    group = ExpertGroup(E, D, H, 50, K, W.clone().to(dev), torch.full((E, D), 1e-6, device=dev), name="up")
    mat = Matrix(40, H, 7, Wd.clone().to(dev), torch.full((40,), 1e-6, device=dev))
    grad = gains.clone().to(dev)
    st = Step([mat], R, T, B.LOGRA_BF16, groups=[group], grads=[grad])
    Wb = W.to(torch.bfloat16).to(dev)
    made, ref = [], dict(S=np.zeros((E, D, R)), Sd=np.zeros((40, R)))
    for mb in range(MBS):
        ids, w, X, dY = _layer(dev, mb)
        d_ids, d_w, d_X, d_dY = ids.to(dev), w.to(dev).contiguous(), X.to(dev), dY.to(dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        order = torch.empty(T * K, dtype=torch.int32, device=dev)
        slots = torch.empty(T, K, dtype=torch.int32, device=dev)
        L.logra_expert_sort(d_ids, E, offsets, order, slots)
        Xs = torch.zeros(T * K, H, dtype=torch.bfloat16, device=dev)
        L.logra_expert_gather(d_X, slots, Xs)
        bounds = offsets.tolist()
        Ys = torch.zeros(T * K, D, dtype=torch.bfloat16, device=dev)
        for e in range(E):
            Ys[bounds[e]:bounds[e + 1]] = Xs[bounds[e]:bounds[e + 1]] @ Wb[e].t()
        Y = torch.empty(T, D, dtype=torch.bfloat16, device=dev)
        L.logra_expert_combine(Ys, slots, Y, weights=d_w)
        dYs = torch.zeros(T * K, D, dtype=torch.bfloat16, device=dev)
        dw = torch.empty(T, K, device=dev)
        L.logra_expert_combine_backward(d_dY, Ys, slots, d_w, dYs, dw)
        dXs = torch.zeros(T * K, H, dtype=torch.bfloat16, device=dev)
        for e in range(E):
            dXs[bounds[e]:bounds[e + 1]] = dYs[bounds[e]:bounds[e + 1]] @ Wb[e]
        dX = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        L.logra_expert_combine(dXs, slots, dX)
        dYd = d_dY[:, :40]
        made.append((d_X, dYs, offsets, order, dYd.contiguous()))

        # the same in fp64, token by token
        W64, x, gy, w64 = to_f64(Wb), to_f64(X), to_f64(dY), to_f64(w)
        y, dx, dwr, G = np.zeros((T, D)), np.zeros((T, H)), np.zeros((T, K)), np.zeros((E, D, H))
        for t in range(T):
            for j in range(K):
                e = int(ids[t, j])
                if e >= 0:
                    out = W64[e] @ x[t]
                    y[t] += w64[t, j] * out
                    dwr[t, j] = gy[t] @ out
                    dx[t] += W64[e].T @ (w64[t, j] * gy[t])
                    G[e] += np.outer(w64[t, j] * gy[t], x[t])
        assert rownorm_err(to_f64(Y), y) < BF16_TOL and rownorm_err(to_f64(dX), dx) < BF16_TOL
        scale = np.abs(gy) @ np.ones((D, 1)) * np.abs(y).max()
        assert np.all(np.abs(to_f64(dw) - dwr) <= BF16_TOL * np.maximum(np.abs(dwr), scale))
        for e in range(E):
            ref["S"][e] += G[e] @ oracle.sign_matrix(0, 3, 50 + e, R, H).T
        ref["Sd"] += (gy[:, :40].T @ x) @ oracle.sign_matrix(0, 3, 7, R, H).T

    st.sketch(3, MBS, lambda i, mb: (made[mb][0], made[mb][4]), expert_inputs=lambda i, mb: made[mb][:4])
    torch.cuda.synchronize()
    for e in range(E):
        assert rownorm_err(to_f64(group.S[e]), ref["S"][e]) < BF16_TOL
    assert rownorm_err(to_f64(mat.S), ref["Sd"]) < BF16_TOL
    before = [to_f64(m.S) for m in st.mats] + [to_f64(grad)]
    norm, coef = st.clip(max_norm)
    n_ref, c_ref, scaled = ox.clip(before, max_norm)
    assert abs(norm.item() - n_ref) <= 2.0 ** -23 * n_ref and abs(coef.item() - c_ref) <= 2.0 ** -22 * c_ref
    assert (coef.item() < 1) == (max_norm < 1)
    for m, r in zip([m.S for m in st.mats] + [grad], scaled):
        assert np.all(np.abs(to_f64(m) - r) <= 2.0 ** -22 * np.abs(r) + 1e-40)
    S_ref = [ref["Sd"]] + list(ref["S"])
    _, _, S_ref = ox.clip(S_ref + [to_f64(gains)], max_norm)

    st.pass1(BETA2, EPS)
    q = st.sqnorms()
    assert len(q) == 1 + E and np.all(np.isfinite(q))
    assert st.pass2(LR, [0.5] * len(st.mats), EPS) == 1 + E
    torch.cuda.synchronize()
    for i, m in enumerate(st.mats):
        A = oracle.sign_matrix(0, 3, 7 if i == 0 else 50 + i - 1, R, H)
        W_old = to_f64(Wd if i == 0 else W[i - 1])
        out = oracle.rowadam_rows(S_ref[i], A, np.full(m.d, f32(1e-6)), W_old, beta2=f32(BETA2), eps=f32(EPS),
                                  lr=f32(LR), scale=0.5)
        assert rel_err(to_f64(m.v), out["v_new"]) < 2 * BF16_TOL          # squares: twice the tolerance of S
        assert w_update_err(to_f64(m.W), out["W_new"], W_old) < BF16_TOL
        assert abs(q[i] / out["sqnorm"] - 1) < BF16_TOL
    assert torch.equal(group.W[2], group.members[2].W) and not torch.equal(group.W[2].cpu(), W[2])


def test_step_refuses_what_does_not_fit():
    dev = device()
    with pytest.raises(ValueError):
        Step([], R, T, B.LOGRA_BF16)
    with pytest.raises(ValueError):
        Step([], R, T, B.LOGRA_BF16, groups=[ExpertGroup(E, D, H, 0, K, torch.zeros(E, D, H + 8, device=dev),
                                                          torch.zeros(E, D, device=dev))])
    group = ExpertGroup(E, D, H, 0, K, torch.zeros(E, D, H, device=dev), torch.zeros(E, D, device=dev))
    st = Step([], R, T, B.LOGRA_BF16, groups=[group])
    X, dY = torch.zeros(T, H, device=dev).bfloat16(), torch.zeros(T * K - 1, D, device=dev).bfloat16()
    offsets, order = torch.zeros(E + 1, dtype=torch.int32, device=dev), torch.zeros(T * K - 1, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        st.sketch(0, 1, expert_inputs=lambda i, mb: (X, dY, offsets, order))


def test_clip_captured_at_once_and_with_a_replaced_gradient():
    """The first clip of a step may be a captured one, and a gradient that the
    caller puts in another's place is the one clipped from then on."""
    dev = device()
    side = torch.cuda.Stream(device=dev)
    g = torch.Generator().manual_seed(31)
    mat = Matrix(40, H, 7, torch.zeros(40, H, device=dev), torch.zeros(40, device=dev))
    first, second = torch.zeros(H + 1, device=dev), torch.randn(2 * H, generator=g).to(dev)
    with torch.cuda.stream(side):
        st = Step([mat], R, T, B.LOGRA_BF16, grads=[first])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm, coef = st.clip(0.5)
    for scale in (1.0, 1e-4, 3.0):
        S, d = torch.randn(40, R, generator=g) * scale, torch.randn(H + 1, generator=g) * scale
        mat.S.copy_(S)
        first.copy_(d)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        n_ref, c_ref, out = ox.clip([to_f64(S), to_f64(d)], 0.5)
        assert abs(norm.item() - n_ref) <= 2.0 ** -23 * n_ref and abs(coef.item() - c_ref) <= 2.0 ** -22 * c_ref
        for got, want in zip((mat.S, first), out):
            assert np.all(np.abs(to_f64(got) - want) <= 2.0 ** -22 * np.abs(want))
    kept, st.grads[0] = first.clone(), second
    n_ref, c_ref, out = ox.clip([to_f64(mat.S), to_f64(second)], 0.5)
    norm, coef = st.clip(0.5)
    torch.cuda.synchronize()
    assert abs(norm.item() - n_ref) <= 2.0 ** -23 * n_ref and torch.equal(first, kept)
    for got, want in zip((mat.S, second), out):
        assert np.all(np.abs(to_f64(got) - want) <= 2.0 ** -22 * np.abs(want))
