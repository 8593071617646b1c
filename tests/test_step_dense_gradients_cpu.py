"""The dense update takes gradients that this step's clip took, on the CPU with
stand-ins for the library's calls: a gradient put in another's place in the
step's list is what is clipped from then on, so an AdamW list that has the old
one is refused, not run on a gradient that nobody writes or clips."""
import pytest
import torch

from test_step_cpu import sim  # noqa: F401
from test_step_dense_cpu import FakeAdamW, _step

HYPER = (1e-3, 0.9, 0.99, 1e-8, 0.1, 7)


@pytest.mark.parametrize("captured", [False, True])
def test_a_replaced_gradient(sim, monkeypatch, captured):  # noqa: F811
    a, b = torch.zeros(3), torch.zeros(4)
    st, _, calls = _step(sim, monkeypatch, grads=[a, b], own=[torch.zeros(5)])
    sim.capturing = captured
    st.clip(1.0)
    sim.capturing = False
    st.dense_update(*HYPER)
    new = torch.zeros(4)
    st.grads[[g is b for g in st.grads].index(True)] = new
    st.clip(1.0)
    n = len(calls)
    with pytest.raises(ValueError):
        st.dense_update(*HYPER)
    assert len(calls) == n
    st.adamw = FakeAdamW([a, new])              # listed anew, as clip lists it
    st.dense_update(*HYPER)
    assert calls[-1][0] == "adamw"


def test_gradients_that_nothing_clips(sim, monkeypatch):  # noqa: F811
    st, _, calls = _step(sim, monkeypatch, grads=[torch.zeros(3)])
    st.grads.clear()
    st.dense_update(*HYPER)
    assert calls[-1][0] == "adamw" and calls[-1][2] is None
