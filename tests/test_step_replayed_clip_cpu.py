"""The dense update after a captured clip, on the CPU with stand-ins for the
library's calls: a graph's replay tells the host nothing, so once a clip was
captured the update always reads the norm, and a sketch sets it back so that an
earlier step's has no say."""
import pytest
import torch

from rank_gradient_sketching_sketch_amd import binding as B
from test_step_cpu import sim  # noqa: F401
from test_step_dense_cpu import _Rows, _step

HYPER = (1e-3, 0.9, 0.99, 1e-8, 0.1, 7)


def _sketch(st):
    st.sketch(2, 1, lambda i, mb: (_Rows(), _Rows()))


@pytest.mark.parametrize("whole", [False, True])
def test_update_after_a_replay(sim, monkeypatch, whole):  # noqa: F811
    st, _, calls = _step(sim, monkeypatch, grads=[torch.zeros(3)])

    def norm():
        st.dense_update(*HYPER)
        return calls[-1][2]

    sim.capturing = True
    if whole:
        _sketch(st)
    st.clip(1.0)
    sim.capturing = False
    for _ in range(3):                  # eager sketch, replayed clip (which writes the norm), eager update
        if not whole:
            _sketch(st)
            assert float(st.norm) == 0.0
        st.norm.fill_(float("nan"))
        assert norm() is st.norm and bool(torch.isnan(st.norm))
    _sketch(st)                         # not clipped at all
    assert norm() is st.norm and float(st.norm) == 0.0


def test_a_captured_sketch_sets_the_norm_back(sim, monkeypatch):  # noqa: F811
    """It may have been captured before any clip was."""
    st, _, _ = _step(sim, monkeypatch, grads=[torch.zeros(3)])
    st.norm.fill_(float("nan"))
    sim.capturing = True
    _sketch(st)
    assert float(st.norm) == 0.0


def test_eager_clips_norm_stays(sim, monkeypatch):  # noqa: F811
    """Without a captured clip the norm that clip returned is there until the next one."""
    st, _, _ = _step(sim, monkeypatch, grads=[torch.zeros(3)])
    norm, _ = st.clip(1.0)
    norm.fill_(4.0)
    _sketch(st)
    assert float(norm) == 4.0
