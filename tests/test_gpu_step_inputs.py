"""Inputs that the step's callbacks make when they are asked for them: the
microbatch's router, sort and gradients run on the caller's stream inside
`Step.sketch`, whose calls are spread over several streams. The sketches are
the same bits as with inputs that were there before."""
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from rank_gradient_sketching_sketch_amd import binding as B
from rank_gradient_sketching_sketch_amd.step import ExpertGroup, Matrix, Step
from gpu_util import device, say

pytestmark = pytest.mark.gpu

T, K, E, D, H, R, MBS = 160, 2, 5, 72, 96, 64, 4
WAIT = 1000000         # cycles that the caller's stream is busy before an input is made


def _parts(dev, n_dense, n_groups):
    mats = [Matrix(40 + 8 * i, H, i, torch.zeros(40 + 8 * i, H, device=dev), torch.zeros(40 + 8 * i, device=dev))
            for i in range(n_dense)]
    groups = [ExpertGroup(E, D, H, 100 + E * i, K, torch.zeros(E, D, H, device=dev), torch.zeros(E, D, device=dev))
              for i in range(n_groups)]
    return mats, groups


def _source(dev, st):
    """What the inputs are computed from, per (matrix or group, microbatch)."""
    g = torch.Generator().manual_seed(17)

    def rows(n, h):
        return torch.randn(n, h, generator=g).to(torch.bfloat16).to(dev)

    dense = {(i, mb): (rows(T, H), rows(T, m.d)) for i, m in enumerate(st.dense) for mb in range(MBS)}
    experts = {(i, mb): (rows(T, H), rows(T * K, D), torch.randint(-1, E, (T, K), generator=g).to(dev))
               for i in range(len(st.groups)) for mb in range(MBS)}
    return dense, experts


def _make(dev, dense, experts, wait):
    """The two callbacks; every tensor they return is new and held by nobody else."""
    def new(t):
        old = torch.full_like(t, float("nan"))      # what a block used again too early would show
        del old
        if wait:
            torch.cuda._sleep(WAIT)
        return t * 1

    def inputs(i, mb):
        return tuple(new(t) for t in dense[i, mb])

    def expert_inputs(i, mb):
        X, dY, ids = experts[i, mb]
        if wait:
            torch.cuda._sleep(WAIT)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        order = torch.empty(T * K, dtype=torch.int32, device=dev)
        L.logra_expert_sort(ids, E, offsets, order, torch.empty(T, K, dtype=torch.int32, device=dev))
        return new(X), new(dY), offsets, order

    return inputs, expert_inputs


def _sketches(st):
    return [m.S.clone() for m in st.mats]


@pytest.mark.parametrize("n_dense,n_groups,lanes", [(1, 1, 0), (2, 2, 0), (0, 2, 2), (3, 0, 0), (1, 1, 1)])
def test_inputs_made_on_the_way(n_dense, n_groups, lanes):
    dev = device()
    say("step inputs", n_dense, n_groups, lanes)
    mats, groups = _parts(dev, n_dense, n_groups)
    st = Step(mats, R, T, B.LOGRA_BF16, groups=groups, sketch_lanes=lanes, parts="none")
    dense, experts = _source(dev, st)
    make, make_experts = _make(dev, dense, experts, False)
    ready = {k: make(*k) for k in dense}
    ready_e = {k: make_experts(*k) for k in experts}
    torch.cuda.synchronize()
    st.sketch(2, MBS, lambda i, mb: ready[i, mb], expert_inputs=lambda i, mb: ready_e[i, mb], late=False)
    torch.cuda.synchronize()
    want = _sketches(st)
    assert all(torch.isfinite(S).all() and S.any() for S in want)
    for m in st.mats:
        m.S.fill_(float("nan"))
    make, make_experts = _make(dev, dense, experts, True)
    for late in (True, True) if n_groups == 0 else (None, True):       # None: late if there are groups
        st.sketch(2, MBS, make, expert_inputs=make_experts, late=late)
        torch.cuda.synchronize()
        for got, S in zip(_sketches(st), want):
            assert torch.equal(got, S)
    # the caller on a stream of its own
    side = torch.cuda.Stream(device=dev)
    with torch.cuda.stream(side):
        st.sketch(2, MBS, make, expert_inputs=make_experts, late=True)
    torch.cuda.synchronize()
    for got, S in zip(_sketches(st), want):
        assert torch.equal(got, S)


def test_captured_with_its_inputs():
    dev = device()
    side = torch.cuda.Stream(device=dev)
    with torch.cuda.stream(side):
        mats, groups = _parts(dev, 1, 2)
        st = Step(mats, R, T, B.LOGRA_BF16, groups=groups, parts="none")
        dense, experts = _source(dev, st)
        make, make_experts = _make(dev, dense, experts, True)
        st.sketch(2, MBS, make, expert_inputs=make_experts, late=True)
        torch.cuda.synchronize()
        want = _sketches(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st.sketch(2, MBS, make, expert_inputs=make_experts, late=True)
    for _ in range(3):
        for m in st.mats:
            m.S.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, S in zip(_sketches(st), want):
            assert torch.equal(got, S)
