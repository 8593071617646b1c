"""A clip that was captured in a graph, with the sketch and the dense update
called eagerly around its replays: a norm that is not finite leaves the dense
parameters and their moments as they are, in every step."""
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from rank_gradient_sketching_sketch_amd import binding as B
from rank_gradient_sketching_sketch_amd.step import Matrix, Step
from gpu_util import device

pytestmark = pytest.mark.gpu
T, D, H, R = 32, 40, 64, 32
HYPER = (1e-3, 0.9, 0.99, 1e-8, 0.1)


def _step(dev, bits):
    g = torch.Generator().manual_seed(3)
    p, d = torch.randn(300, generator=g).to(dev), torch.zeros(300, device=dev)
    mat = Matrix(D, H, 7, torch.zeros(D, H, device=dev), torch.zeros(D, device=dev))
    dense = L.AdamWList([p], [d], state_bits=bits)
    return Step([mat], R, T, B.LOGRA_BF16, adamw=dense), dense, p, d


def _bits(dense):
    return [t.clone() for t in [dense.params[0]] + [s.view(torch.uint8) for s in (dense.exp_avg, dense.exp_avg_sq)]]


def _inputs(dev, seed):
    g = torch.Generator().manual_seed(seed)
    X, dY = torch.randn(T, H, generator=g).bfloat16().to(dev), torch.randn(T, D, generator=g).bfloat16().to(dev)
    return lambda i, mb: (X, dY)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("whole", [False, True])
def test_replayed_clip(whole, bits):
    """whole: the sketch is in the graph too."""
    dev = device()
    side = torch.cuda.Stream(device=dev)
    with torch.cuda.stream(side):
        st, dense, p, d = _step(dev, bits)
        st.sketch(0, 1, _inputs(dev, 9))
        st.clip(0.5)
    torch.cuda.synchronize()
    held = _inputs(dev, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        if whole:
            st.sketch(1, 1, held)
        st.clip(0.5)
    applied = 0
    with torch.cuda.stream(side):
        for step, bad in enumerate([None, float("nan"), None, float("inf"), None], 1):
            if not whole:
                st.sketch(step, 1, _inputs(dev, step))
            d.normal_(generator=torch.Generator(device=dev).manual_seed(step))
            if bad is not None:
                d[5] = bad
            before = _bits(dense)
            graph.replay()
            st.dense_update(*HYPER, applied + 1)
            torch.cuda.synchronize()
            assert bool(torch.isfinite(st.norm)) == (bad is None)
            same = [torch.equal(a, b) for a, b in zip(before, _bits(dense))]
            assert same == ([False] * 3 if bad is None else [True] * 3), (step, same)
            applied += bad is None
        # a step that is not clipped: the last one's norm has no say
        d[5] = float("nan")
        graph.replay()
        d.fill_(0.01)
        before = _bits(dense)
        st.sketch(9, 1, _inputs(dev, 9))
        st.dense_update(*HYPER, applied + 1)
        torch.cuda.synchronize()
        assert not torch.equal(before[0], p) and bool(torch.isfinite(p).all())
