"""The gradient list's device table and the streams that read it, on the CPU:
the GPU's parts are stand-ins that record what they are asked for."""
import os
import weakref
from types import SimpleNamespace

import pytest
import torch

from rank_gradient_sketching_sketch_amd import binding as B


class FakeStream:
    def __init__(self, handle, device_index=0, **kw):
        self.cuda_stream, self.device_index = handle, device_index


class FakeTable:
    """The table on the GPU."""

    def __init__(self):
        self.kept = set()

    def data_ptr(self):
        return 0x40000

    def get_device(self):
        return 0

    def record_stream(self, s):
        self.kept.add(s.cuda_stream)


class Storage:
    pass


class Gradient:
    """A contiguous float32 gradient on GPU 0."""
    dtype = torch.float32
    device = torch.device("cuda", 0)

    def __init__(self, ptr, *shape):
        self.ptr, self.shape = ptr, torch.Size(shape)

    def data_ptr(self):
        return self.ptr

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def size(self, i):
        return self.shape[i]

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def untyped_storage(self):
        return Storage()


@pytest.fixture
def gpu(monkeypatch):
    """g.current: the current stream; g.calls: (call, stream) of the library's launching calls."""
    if not os.path.exists(B.LIB_PATH):
        from rank_gradient_sketching_sketch_amd import build_lib
        build_lib.build()
    g = SimpleNamespace(current=FakeStream(5), calls=[])
    lib = B.load_library()
    monkeypatch.setattr(torch.Tensor, "to", lambda t, device: FakeTable())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: g.current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(B, "_current_stream", lambda dev: g.current.cuda_stream)
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    fake = SimpleNamespace(logra_grad_table_bytes=lib.logra_grad_table_bytes,
                           logra_grad_list_pack=lib.logra_grad_list_pack,
                           logra_grad_workspace_bytes=lib.logra_grad_workspace_bytes,
                           logra_grad_norm=lambda *a: g.calls.append(("norm", a[-1])) or 0,
                           logra_grad_clip=lambda *a: g.calls.append(("clip", a[-1])) or 0)
    monkeypatch.setattr(B, "load_library", lambda: fake)
    g.one = lambda: SimpleNamespace(dtype=torch.float32, numel=lambda: 1, get_device=lambda: 0, data_ptr=lambda: 0x9000)
    return g


def _list(at=0x100000):
    return B.GradList([Gradient(at, 3, 4), Gradient(at + 0x1000, 9)])


@pytest.mark.parametrize("as_int", [False, True])
def test_table_is_kept_for_every_stream_that_reads_it(gpu, as_int):
    """A table comes from the stream that was current when the list was made;
    for a call on another one its memory is recorded there."""
    grads = _list()
    B.logra_grad_norm(grads, gpu.one())
    B.logra_grad_clip(grads, 1.0, gpu.one(), gpu.one())
    assert gpu.calls == [("norm", 5), ("clip", 5)] and grads.table.kept <= {5}
    out = _list(0x900000)
    side = FakeStream(7)
    B.logra_grad_clip(grads, 1.0, gpu.one(), gpu.one(), out=out, stream=7 if as_int else side)
    assert gpu.calls[-1] == ("clip", 7)
    assert 7 in grads.table.kept and 7 in out.table.kept
    B.logra_grad_norm(grads, gpu.one(), stream=8 if as_int else FakeStream(8))
    assert 8 in grads.table.kept
    gpu.current = FakeStream(9)                 # no stream named, another one current than at the making
    B.logra_grad_norm(out, gpu.one())
    assert gpu.calls[-1] == ("norm", 9) and 9 in out.table.kept


def test_memory_of_a_listed_tensor_lives_as_long_as_the_list(gpu):
    """A gradient whose storage is exchanged under it (t.data, set_) leaves
    the list's addresses in memory that the list still holds."""
    made = []

    class Counted(Gradient):
        def untyped_storage(self):
            made.append(Storage())
            return made[-1]

    grads = B.GradList([Counted(0x100000, 3, 4), Counted(0x200000, 9)])
    held = [weakref.ref(t) for t in made]
    made.clear()
    assert len(held) == 2 and all(t() is not None for t in held)
    del grads
    assert all(t() is None for t in held)


def test_list_tells_whether_it_describes_its_tensors(gpu):
    """An exchanged storage, another shape, stride or type under the same
    object is another gradient."""
    a, b = Gradient(0x100000, 3, 4), Gradient(0x200000, 9)
    grads = B.GradList([a, b])
    assert grads.describes([a, b])
    assert not grads.describes([a]) and not grads.describes([b, a]) and not grads.describes([a, b, b])
    assert not grads.describes([a, Gradient(0x200000, 9)])          # another object: its memory may go any time
    for change in (dict(ptr=0x300000), dict(shape=torch.Size((3, 3))), dict(shape=torch.Size((12,))),
                   dict(dtype=torch.bfloat16)):
        c = Gradient(0x100000, 3, 4)
        grads = B.GradList([c, b])
        for k, v in change.items():
            setattr(c, k, v)
        assert not grads.describes([c, b])


def test_stream_of_another_gpu_is_refused(gpu):
    """A kernel launched there would run beside its tensors' GPU."""
    grads = _list()
    for call in (lambda **kw: B.logra_grad_norm(grads, gpu.one(), **kw),
                 lambda **kw: B.logra_grad_clip(grads, 1.0, gpu.one(), gpu.one(), **kw)):
        with pytest.raises(B.LograError):
            call(stream=FakeStream(7, device_index=1))
        assert not gpu.calls
        call(stream=FakeStream(7))
        assert gpu.calls.pop()[1] == 7


def test_streams_without_torchs_short_cuts(monkeypatch):
    """The two private functions of torch are short cuts: where it has them no
    more, the public ones say the same."""
    import importlib
    kept = {n: getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice")}
    try:
        for n in kept:
            monkeypatch.delattr(torch._C, n, raising=False)
        fresh = importlib.util.module_from_spec(importlib.util.find_spec(B.__name__))
        fresh.__spec__.loader.exec_module(fresh)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: FakeStream(40 + torch.device("cuda", dev).index))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
        assert fresh._current_stream(1) == 41 and fresh._current_device() == 2
    finally:
        monkeypatch.undo()


def test_size_cache_is_bounded(gpu):
    """One size per token count would grow with every new sequence length."""
    assert B.logra_expert_sort_workspace_bytes.cache_info().maxsize is not None
