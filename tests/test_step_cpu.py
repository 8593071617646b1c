"""The step scheduler's ordering, on the CPU: streams, events and the library's
calls are stand-ins that record which work each stream has waited for."""
import os
import weakref
from types import SimpleNamespace

import pytest
import torch

from rank_gradient_sketching_sketch_amd import binding as B
from rank_gradient_sketching_sketch_amd import step as step_module
from rank_gradient_sketching_sketch_amd.step import ExpertGroup, Matrix, Step

T, K, E, D, H, R = 16, 2, 3, 32, 64, 32


class FakeStream:
    """`seen`: the pieces of work that are over before the stream's next one starts."""
    count = 0

    def __init__(self, device=None, **kw):
        FakeStream.count += 1
        self.cuda_stream, self.device_index = FakeStream.count, 0
        self.seen, self.idle = set(), True

    def work(self, name):
        self.seen.add(name)
        self.idle = False
        return name

    def wait_event(self, e):
        self.seen |= e.seen

    def wait_stream(self, s):
        self.seen |= s.seen

    def query(self):
        return self.idle


class FakeEvent:
    def __init__(self, *a, **kw):
        self.seen = set()

    def record(self, stream):
        self.seen = set(stream.seen)


class FakeTensor:
    """A tensor that work `made` on `stream` writes; `kept` are the streams it was recorded on."""

    def __init__(self, shape, stream, made=None):
        self.shape, self.stream, self.made, self.kept = shape, stream, made, set()

    def record_stream(self, s):
        self.kept.add(s)


@pytest.fixture
def sim(monkeypatch):
    if not os.path.exists(B.LIB_PATH):
        from rank_gradient_sketching_sketch_amd import build_lib
        build_lib.build()
    s = SimpleNamespace(current=[FakeStream()], calls=[], seen=[], capturing=False)

    class Use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            s.current.append(self.stream)

        def __exit__(self, *exc):
            s.current.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: s.current[-1])
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "Event", FakeEvent)
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: s.capturing)
    monkeypatch.setattr(B, "GradList", FakeList)

    def reads(name, st, *tensors):
        for t in tensors:
            if t.made is not None and st is not t.stream:
                assert t.made in st.seen, "%s reads %s before it is there" % (name, t.made)
                assert st in t.kept, "%s is not kept from other use" % t.made
        s.calls.append((name, st))
        s.seen.append(set(st.seen))
        st.work("%s %d" % (name, len(s.calls)))

    monkeypatch.setattr(B, "logra_sketch_project", lambda m, X, ws, st, opts: reads("project", st, X))
    monkeypatch.setattr(B, "logra_sketch_fold", lambda m, dY, S, acc, ws, st, opts: reads("fold", st, dY))
    monkeypatch.setattr(B, "logra_sketch_fold_parts", lambda m, dY, S, parts, phase, ws, st, opts: reads("fold", st, dY))
    monkeypatch.setattr(B, "logra_sketch_experts", lambda m, offsets, X, dY, S, acc, order, topk, ws, stream: reads(
        "experts", stream, *[t for t in (offsets, X, dY, order) if t is not None]))
    return s


def _step(n_dense, n_groups, **kw):
    mats = [Matrix(D, H, i, torch.zeros(D, H), torch.zeros(D)) for i in range(n_dense)]
    groups = [ExpertGroup(E, D, H, 100 + E * i, K, torch.zeros(E, D, H), torch.zeros(E, D)) for i in range(n_groups)]
    return Step(mats, R, T, B.LOGRA_F32, groups=groups, **kw)


def _run(st, sim, made, mbs=3, **kw):
    """One step's sketches whose inputs the callbacks make on the current
    stream (made) or had before."""
    def new(what, shape):
        cur = sim.current[-1]
        return FakeTensor(shape, cur, cur.work(what) if made else None)

    return st.sketch(1, mbs, lambda i, mb: (new("X %d %d" % (i, mb), (T, H)), new("dY %d %d" % (i, mb), (T, D))),
                     expert_inputs=lambda g, mb: (new("Xe %d %d" % (g, mb), (T, H)), new("dYe %d %d" % (g, mb), (T * K, D)),
                                                  new("offsets %d %d" % (g, mb), (E + 1,)),
                                                  new("order %d %d" % (g, mb), (T * K,)) if g == 0 else None), **kw)


@pytest.mark.parametrize("dense,groups,kw", [(1, 1, {}), (0, 2, {}), (3, 2, {}), (0, 1, {}), (1, 0, dict(late=True)),
                                             (5, 0, dict(late=True))])
@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("capturing", [False, True])
def test_inputs_made_in_the_callbacks_are_waited_for(sim, dense, groups, kw, other, capturing):
    """What a callback enqueues on the caller's stream is over before a lane
    reads it, and its memory is kept; `other`: the caller's stream is not the
    one that the step was made on."""
    st = _step(dense, groups)
    if other:
        sim.current.append(FakeStream())
    sim.capturing = capturing
    _run(st, sim, True, **kw)
    for name, lane in sim.calls:
        assert any(lane is ln["stream"] for ln in st.lanes)
    lanes = {id(ln["stream"]): ln["stream"] for ln in st.lanes}.values()
    for ln in lanes:
        assert ln.seen <= st.main.seen              # joined
    assert len(sim.calls) == 3 * (2 * dense + groups)


@pytest.mark.parametrize("dense,groups,kw", [(3, 1, {}), (0, 3, {}), (3, 1, dict(late=False)), (4, 0, {})])
def test_inputs_made_before_leave_the_lanes_apart(sim, dense, groups, kw):
    """Callbacks that enqueue nothing make no lane wait for another."""
    st = _step(dense, groups)
    sim.current[-1].idle = True
    _run(st, sim, False, **kw)
    lanes = [lane for _, lane in sim.calls]
    assert len({id(lane) for lane in lanes}) == st.n_sketch > 2
    for i, (lane, seen) in enumerate(zip(lanes, sim.seen)):
        for j, (name, other) in enumerate(sim.calls[:i]):
            assert ("%s %d" % (name, j + 1) in seen) == (other is lane)


@pytest.mark.parametrize("late", [False, True])
def test_a_callback_that_fails_leaves_no_lane_unjoined(sim, late):
    """Work that was enqueued before an exception is over before what the
    caller does next."""
    for wrong in ("raise", "rows"):
        st = _step(3, 1)

        def inputs(i, mb):
            if wrong == "raise" and mb == 1 and i == 2:
                raise RuntimeError("no more rows")
            cur = sim.current[-1]
            return FakeTensor((T, H), cur, cur.work("X") if late else None), FakeTensor((T, D), cur)

        def experts(g, mb):
            return tuple(FakeTensor((T * K - (mb == 1), D), sim.current[-1]) for _ in range(4))

        with pytest.raises((RuntimeError, ValueError)):
            st.sketch(1, 3, inputs, expert_inputs=experts, late=late)
        for ln in st.lanes:
            assert ln["stream"].seen <= st.main.seen
        assert st.callbacks is None or st.callbacks.seen <= st.main.seen
        assert sim.current == [st.main]


class FakeList:
    """Stands for a gradient list: alive as long as somebody holds it."""

    def __init__(self, tensors, device=None):
        self.tensors, self.workspace_bytes = list(tensors), 0

    def describes(self, tensors):
        return len(tensors) == len(self.tensors) and all(a is b for a, b in zip(self.tensors, tensors))


def test_list_that_a_graph_reads_outlives_a_replaced_gradient(sim, monkeypatch):
    """A captured clip's table and workspace stay when a later clip lists
    other gradients: the graph still reads them at every replay. Lists that no
    graph reads go."""
    monkeypatch.setattr(B, "GradList", FakeList)
    seen = []
    monkeypatch.setattr(B, "logra_grad_clip", lambda lst, *a, ws, stream: seen.append((weakref.ref(lst), weakref.ref(ws))))
    mats = [Matrix(D, H, 0, torch.zeros(D, H), torch.zeros(D))]
    st = Step(mats, R, T, B.LOGRA_F32, grads=[torch.zeros(7)])
    sim.capturing = True
    st.clip(1.0)
    st.clip(1.0)
    sim.capturing = False
    for n in (5, 9, 11):
        st.grads[0] = torch.zeros(n)
        st.clip(1.0)
    alive = [lst() is not None for lst, _ in seen]
    assert alive == [True, True, False, False, True]
    assert [ws() is not None for _, ws in seen] == alive
    sim.capturing = True                # the last list too, from now on
    st.clip(1.0)
    sim.capturing = False
    st.grads[0] = torch.zeros(3)
    st.clip(1.0)
    assert seen[-2][0]() is not None and seen[-1][0]() is not None


def test_clip_that_would_list_anew_is_refused_in_a_capture(sim, monkeypatch):
    """Listing copies a table to the GPU, which a capture cannot."""
    monkeypatch.setattr(B, "GradList", FakeList)
    monkeypatch.setattr(B, "logra_grad_clip", lambda *a, **kw: None)
    st = Step([Matrix(D, H, 0, torch.zeros(D, H), torch.zeros(D))], R, T, B.LOGRA_F32, grads=[torch.zeros(7)])
    st.grads[0] = torch.zeros(8)
    sim.capturing = True
    with pytest.raises(ValueError):
        st.clip(1.0)
    sim.capturing = False
    st.clip(1.0)
    sim.capturing = True
    st.clip(1.0)


def test_clip_lists_anew_when_a_storage_was_exchanged(sim, monkeypatch):
    """Same object, other memory: the list made before does not describe it."""
    class List(FakeList):
        def __init__(self, tensors, device=None):
            super().__init__(tensors)
            self.ptrs = [t.data_ptr() for t in self.tensors]

        def describes(self, tensors):
            return len(tensors) == len(self.ptrs) and all(
                a is b and b.data_ptr() == p for a, b, p in zip(self.tensors, tensors, self.ptrs))

    monkeypatch.setattr(B, "GradList", List)
    seen = []
    monkeypatch.setattr(B, "logra_grad_clip", lambda lst, *a, ws, stream: seen.append(lst.ptrs))
    grad = torch.zeros(7)
    st = Step([Matrix(D, H, 0, torch.zeros(D, H), torch.zeros(D))], R, T, B.LOGRA_F32, grads=[grad])
    st.clip(1.0)
    grad.data = torch.ones(7)
    st.clip(1.0)
    st.mats[0].S.set_(torch.zeros(D, R))
    st.clip(1.0)
    assert [p[1] for p in seen[1:]] == [grad.data_ptr()] * 2 and seen[0] != seen[1] != seen[2]
    assert seen[2][0] == st.mats[0].S.data_ptr()


def test_members_sketches_are_the_groups(sim, monkeypatch):
    """The experts' S are views of their group's: one put in its place (or its
    storage exchanged) is what every phase uses; a member's alone is refused."""
    monkeypatch.setattr(B, "logra_grad_clip", lambda *a, **kw: None)
    used = []
    monkeypatch.setattr(B, "logra_update_sqnorm_batch",
                        lambda descs, code, S, *a: used.append([t.data_ptr() for t in S]))
    monkeypatch.setattr(B, "logra_rowadam_apply", lambda desc, code, S, *a, **kw: used.append([S.data_ptr()]))
    st = _step(0, 1, apply_lanes=1)
    group = st.groups[0]

    def phases():
        _run(st, sim, False)
        st.clip(1.0)
        for phase in (lambda: st.pass1(0.9, 1e-8), lambda: st.pass2(1e-3, [1.0] * E, 1e-8)):
            used.clear()
            phase()
            assert [p for call in used for p in call] == [group.S[e].data_ptr() for e in range(E)]

    phases()
    for other in (lambda: setattr(group, "S", torch.zeros(E, D, R)), lambda: group.S.set_(torch.zeros(E, D, R)),
                  lambda: setattr(group.S, "data", torch.zeros(E, D, R))):
        old = [m.S.data_ptr() for m in group.members]
        other()
        st.pass1(0.9, 1e-8)                 # whichever phase comes first
        phases()
        assert old != [m.S.data_ptr() for m in group.members]
    good = group.S
    for bad in (torch.zeros(E, D, R + 1), torch.zeros(E, D, R, dtype=torch.float64), torch.zeros(E, R, D).transpose(1, 2)):
        group.S = bad
        for phase in (lambda: _run(st, sim, False), lambda: st.clip(1.0), lambda: st.pass1(0.9, 1e-8),
                      lambda: st.pass2(1e-3, [1.0] * E, 1e-8)):
            with pytest.raises(ValueError):
                phase()
    group.S = good
    phases()
    mine = group.members[1].S
    group.members[1].S = torch.zeros(D, R)
    for phase in (lambda: _run(st, sim, False), lambda: st.clip(1.0), lambda: st.pass1(0.9, 1e-8),
                  lambda: st.pass2(1e-3, [1.0] * E, 1e-8)):
        with pytest.raises(ValueError):
            phase()
    group.members[1].S = mine
    phases()


def test_second_step_of_a_group_goes_on_where_the_first_left(sim, monkeypatch):
    """A group given to another Step keeps its experts' state: v is what the
    last update left, not what the group was made with."""
    monkeypatch.setattr(B, "logra_update_sqnorm_batch", lambda *a, **kw: None)
    monkeypatch.setattr(B, "logra_rowadam_apply", lambda *a, **kw: None)
    group = ExpertGroup(E, D, H, 100, K, torch.zeros(E, D, H), torch.zeros(E, D))
    first = Step([], R, T, B.LOGRA_F32, groups=[group], apply_lanes=1)
    first.set_step(1)
    first.pass2(1e-3, [1.0, None, 1.0], 1e-8)
    now = [m.v.data_ptr() for m in group.members]
    assert now[0] != group.v[0].data_ptr() and now[1] == group.v[1].data_ptr()
    second = Step([], R, 2 * T, B.LOGRA_F32, groups=[group], apply_lanes=1)
    assert [m.v.data_ptr() for m in second.mats] == now
    assert [m.W.data_ptr() for m in second.mats] == [group.W[e].data_ptr() for e in range(E)]
    second.set_step(2)
    for st in (first, second):
        st.pass1(0.9, 1e-8)
        assert [m.S.data_ptr() for m in st.mats] == [group.S[e].data_ptr() for e in range(E)]
    # state put in the group's place, and other memory under it, is what the next phase uses
    for what, new in (("v", lambda: setattr(group, "v", torch.ones(E, D))),
                      ("v", lambda: setattr(group.v, "data", torch.ones(E, D))),
                      ("W", lambda: setattr(group, "W", torch.ones(E, D, H))), ("W", lambda: group.W.set_(torch.ones(E, D, H)))):
        new()
        first.pass1(0.9, 1e-8)
        for st in (first, second):
            assert [getattr(m, what).data_ptr() for m in st.mats] == [getattr(group, what)[e].data_ptr() for e in range(E)]
    group.v = torch.ones(E, D + 1)
    with pytest.raises(ValueError):
        first.pass1(0.9, 1e-8)
