"""The step's dense parameters, on the CPU with stand-ins for the library's
calls: their gradients are clipped with the sketches, and the update takes the
norm of this step's clipping, and of this step's alone."""
import pytest
import torch

from rank_gradient_sketching_sketch_amd import binding as B
from rank_gradient_sketching_sketch_amd.step import Matrix, Step
from test_step_cpu import D, H, R, T, FakeList, sim  # noqa: F401


class FakeAdamW:
    def __init__(self, grads):
        self.params, self.grads, self.copies = [torch.zeros_like(g) for g in grads], list(grads), [None] * len(grads)
        self.whole = True

    def describes(self, params, grads, copies=None):
        return self.whole and params is self.params and grads is self.grads


def _step(sim, monkeypatch, grads=(), own=()):
    calls = []
    monkeypatch.setattr(B, "GradList", FakeList)
    monkeypatch.setattr(B, "logra_grad_clip", lambda lst, *a, ws, stream: calls.append(("clip", lst.tensors)))
    monkeypatch.setattr(B, "logra_adamw", lambda lst, *a, norm, seed, stream: calls.append(("adamw", a, norm, seed, stream)))
    adamw = FakeAdamW(grads)
    return Step([Matrix(D, H, 0, torch.zeros(D, H), torch.zeros(D))], R, T, B.LOGRA_F32, grads=own, adamw=adamw, seed=5), adamw, calls


def test_gradients_are_clipped_once(sim, monkeypatch):  # noqa: F811
    a, b, c = torch.zeros(3), torch.zeros(4), torch.zeros(5)
    st, _, calls = _step(sim, monkeypatch, grads=[a, b], own=[b, c])
    st.clip(1.0)
    listed = calls[0][1]
    assert [sum(t is g for t in listed) for g in (a, b, c)] == [1, 1, 1] and listed[0] is st.mats[0].S


def test_update_takes_the_norm_of_its_own_step(sim, monkeypatch):  # noqa: F811
    st, _, calls = _step(sim, monkeypatch, grads=[torch.zeros(3)])
    hyper = (1e-3, 0.9, 0.99, 1e-8, 0.1, 7)
    st.dense_update(*hyper)                                      # not clipped
    st.clip(1.0)
    st.dense_update(*hyper)
    st.sketch(2, 1, lambda i, mb: (_Rows(), _Rows()))            # the next step, not clipped
    st.dense_update(*hyper)
    updates = [c for c in calls if c[0] == "adamw"]
    assert [u[1] for u in updates] == [hyper] * 3 and all(u[3] == 5 and u[4] is st.main for u in updates)
    assert updates[0][2] is None and updates[1][2] is st.norm and updates[2][2] is None


class _Rows:
    shape, made, stream = (T, H), None, None


def test_refusals(sim, monkeypatch):  # noqa: F811
    st, adamw, _ = _step(sim, monkeypatch, grads=[torch.zeros(3)])
    adamw.whole = False
    with pytest.raises(ValueError):
        st.dense_update(1e-3, 0.9, 0.99, 1e-8, 0.1, 1)
    bare = Step([Matrix(D, H, 0, torch.zeros(D, H), torch.zeros(D))], R, T, B.LOGRA_F32)
    with pytest.raises(ValueError):
        bare.dense_update(1e-3, 0.9, 0.99, 1e-8, 0.1, 1)
