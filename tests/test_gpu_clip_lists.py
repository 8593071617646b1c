"""What may happen to a gradient list around a call: dropped while another
stream still reads its table, listed anew under a captured graph. What a table's memory is used for next here is
another valid table, whose tensors would show a call that reads it too early."""
import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from oracle import experts as ox
from rank_gradient_sketching_sketch_amd import binding as B
from rank_gradient_sketching_sketch_amd.step import Matrix, Step
from gpu_util import device, say, to_f64

pytestmark = pytest.mark.gpu


def _tensors(dev, seed, n=80, size=1700):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(size + i, generator=g).to(dev) for i in range(n)]


@pytest.mark.parametrize("current", [False, True])
def test_list_dropped_under_a_call_on_another_stream(current):
    dev = device()
    say("list dropped", current)
    grads = _tensors(dev, 1)
    outs = [torch.zeros_like(t) for t in grads]
    decoys = [torch.full_like(t, 5.0) for t in grads]
    glist, other = L.GradList(grads), L.GradList(decoys)
    norm, coef = torch.zeros(1, device=dev), torch.zeros(1, device=dev)
    L.logra_grad_clip(glist, 3.0, norm, coef, out=L.GradList(outs))
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream(device=dev)
    for _ in range(3):
        for t in outs:
            t.zero_()
        out = L.GradList(outs)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(5000000)
            if current:
                L.logra_grad_clip(glist, 3.0, norm, coef, out=out)
        if not current:
            L.logra_grad_clip(glist, 3.0, norm, coef, out=out, stream=side)
        del out
        later = [other.table.clone() for _ in range(8)]
        torch.cuda.synchronize()
        del later
        for got, ref, d in zip(outs, want, decoys):
            assert torch.equal(got, ref) and (d == 5.0).all()


def test_graph_of_a_clip_whose_gradient_was_replaced():
    """The graph goes on clipping the tensors of its capture, with the table
    and the workspace it was captured with."""
    dev = device()
    say("replaced under a graph")
    D, R, H = 900, 64, 96                       # enough elements for a workspace
    side = torch.cuda.Stream(device=dev)
    mat = Matrix(D, H, 7, torch.zeros(D, H, device=dev), torch.zeros(D, device=dev))
    g = torch.Generator().manual_seed(31)
    first, second = torch.zeros(1500, device=dev), torch.randn(1500, generator=g).to(dev)
    with torch.cuda.stream(side):
        st = Step([mat], R, 200, B.LOGRA_BF16, grads=[first])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm, coef = st.clip(0.5)
    torch.cuda.synchronize()

    def fill(scale):
        mat.S.copy_(torch.randn(D, R, generator=g) * scale)
        first.copy_(torch.randn(1500, generator=g) * scale)
        torch.cuda.synchronize()

    def replay():
        grads = [to_f64(mat.S), to_f64(first)]
        graph.replay()
        torch.cuda.synchronize()
        n_ref, c_ref, out = ox.clip(grads, 0.5)
        assert abs(norm.item() - n_ref) <= 2.0 ** -23 * n_ref and abs(coef.item() - c_ref) <= 2.0 ** -22 * c_ref
        for got, want in zip((mat.S, first), out):
            assert np.all(np.abs(to_f64(got) - want) <= 2.0 ** -22 * np.abs(want))

    fill(1.0)
    replay()
    st.grads[0] = second
    n_ref, _, _ = ox.clip([to_f64(mat.S), to_f64(second)], 0.5)
    norm, coef = st.clip(0.5)
    torch.cuda.synchronize()
    assert abs(norm.item() - n_ref) <= 2.0 ** -23 * n_ref
    kept = second.clone()
    spare = [L.GradList([torch.full((64,), 5.0, device=dev), torch.full((32,), 5.0, device=dev)]) for _ in range(8)]
    for scale in (3.0, 1e-4, 2.0):
        fill(scale)
        replay()
        assert torch.equal(second, kept)
        fill(scale)
        n_ref, _, _ = ox.clip([to_f64(mat.S), to_f64(second)], 1e9)
        st.clip(1e9)
        torch.cuda.synchronize()
        assert abs(norm.item() - n_ref) <= 2.0 ** -23 * n_ref
    assert all((t == 5.0).all() for s in spare for t in s.tensors)


def test_step_whose_gradients_storage_is_exchanged():
    """t.data = and set_ under the same object: the new memory is what is
    clipped, the old one is left as it was."""
    dev = device()
    say("exchanged storage")
    D, R, H = 40, 64, 96
    g = torch.Generator().manual_seed(8)

    def new(*shape):
        return torch.randn(*shape, generator=g).to(dev)

    mat, grad = Matrix(D, H, 7, torch.zeros(D, H, device=dev), torch.zeros(D, device=dev)), new(300)
    st = Step([mat], R, 200, B.LOGRA_BF16, grads=[grad])

    def check():
        grads = [to_f64(mat.S), to_f64(grad)]
        n_ref, _, out = ox.clip(grads, 0.5)
        norm, _ = st.clip(0.5)
        torch.cuda.synchronize()
        assert abs(norm.item() - n_ref) <= 2.0 ** -23 * n_ref
        for got, want in zip((mat.S, grad), out):
            assert np.all(np.abs(to_f64(got) - want) <= 2.0 ** -22 * np.abs(want))

    mat.S.copy_(new(D, R))
    check()
    for exchange in (lambda: setattr(grad, "data", new(300)), lambda: setattr(grad, "data", new(17, 20)),
                     lambda: grad.set_(new(5)), lambda: mat.S.set_(new(D, R))):
        old = (grad.detach(), mat.S.detach())
        kept = [t.clone() for t in old]
        exchange()
        now = {grad.data_ptr(), mat.S.data_ptr()}
        if mat.S.data_ptr() == old[1].data_ptr():
            mat.S.copy_(new(D, R))
        check()
        for t, k in zip(old, kept):
            assert t.data_ptr() in now or torch.equal(t, k)
