"""Host-side checks of routing, 8-bit products and AdamW: every refusal
returns before any launch, and the packed AdamW table. No GPU."""
import ctypes
import os

import numpy as np
import pytest
import torch

FAKE, FAKE2, FAKE3 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10002)
EIGHT = ctypes.c_void_p(0x10008)
OK, BAD, UNSUP, WS = 0, 1, 2, 3
BIG = 1 << 40


@pytest.fixture(scope="module")
def B():
    from rank_gradient_sketching_sketch_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from rank_gradient_sketching_sketch_amd import build_lib
        build_lib.build()
    binding.load_library()
    return binding


def _with(call, base):
    def run(**kw):
        return call(*{**base, **kw}.values())
    return run


def test_route_refusals(B):
    lib = B.load_library()
    f = _with(lib.logra_route, dict(T=4, E=8, K=2, dtype=0, x=FAKE, ld=8, score=0, bias=None, groups=1, kept=1, best=1,
                                    renorm=1, scale=1.0, ids=FAKE2, w=FAKE3, stream=None))
    for kw in (dict(T=-1), dict(E=0), dict(K=0), dict(K=9), dict(score=2), dict(score=-1), dict(x=None), dict(x=HALF),
               dict(ld=7), dict(ids=None), dict(ids=HALF), dict(w=None), dict(w=ODD), dict(bias=HALF), dict(groups=0),
               dict(groups=3), dict(groups=4, kept=0), dict(groups=4, kept=5), dict(best=0), dict(best=3)):
        assert f(**kw) == BAD, kw
    for kw in (dict(dtype=2), dict(E=1025, ld=1025), dict(E=200, ld=200, K=65), dict(T=(1 << 23) + 1), dict(ld=BIG + 1),
               dict(E=130, ld=130, groups=65)):
        assert f(**kw) == UNSUP, kw
    assert f(T=0, x=None, ids=None, w=None) == OK
    b = _with(lib.logra_route_backward, dict(T=4, E=8, K=2, dtype=1, x=FAKE, ld=8, score=1, ids=FAKE2, dw=FAKE3, renorm=0,
                                             scale=1.0, dx=FAKE, ldd=8, stream=None))
    for kw in (dict(T=-1), dict(E=0), dict(K=9), dict(score=7), dict(x=None), dict(x=ODD), dict(ld=7), dict(ids=None),
               dict(dw=None), dict(dw=HALF), dict(dx=None), dict(dx=ODD), dict(ldd=7)):
        assert b(**kw) == BAD, kw
    for kw in (dict(dtype=5), dict(E=1025, ld=1025, ldd=1025), dict(ldd=BIG + 1)):
        assert b(**kw) == UNSUP, kw
    assert b(T=0, x=None, ids=None, dw=None, dx=None) == OK


def test_quantize_refusals(B):
    f = _with(B.load_library().logra_fp8_quantize, dict(batch=1, rows=4, cols=40, dtype=1, x=FAKE, ldx=40, block=1, turned=0,
                                                        codes=FAKE2, ldc=40, scales=FAKE3, stream=None))
    for kw in (dict(batch=-1), dict(rows=-1), dict(cols=-1), dict(block=64), dict(turned=1), dict(x=None), dict(x=ODD),
               dict(ldx=39), dict(codes=None), dict(ldc=39), dict(scales=None), dict(scales=HALF),
               dict(block=128, turned=1, rows=41, ldc=40)):
        assert f(**kw) == BAD, kw
    for kw in (dict(dtype=3), dict(rows=BIG, ldx=BIG), dict(batch=1 << 36, rows=1 << 10), dict(rows=1 << 30, cols=1 << 10, ldx=1 << 10, ldc=1 << 10),
               dict(cols=1 << 31, ldx=1 << 31, ldc=1 << 31)):
        assert f(**kw) == UNSUP, kw
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0, ldx=0)):
        assert f(**{**kw, "x": None, "codes": None, "scales": None}) == OK, kw


def test_matmul_refusals(B):
    f = _with(B.load_library().logra_fp8_matmul, dict(M=4, n=8, k=32, E=1, offsets=None, order=None, topk=1, x=FAKE, ldx=32, rows=4,
                                                      xs=FAKE, w=FAKE2, ldw=32, ws=FAKE2, dtype=1, y=FAKE3, ldy=8, stream=None))
    for kw in (dict(M=-1), dict(n=0), dict(k=0), dict(E=0), dict(E=2), dict(rows=3), dict(rows=-1), dict(order=FAKE), dict(x=None),
               dict(x=EIGHT), dict(ldx=16), dict(ldx=40), dict(xs=None), dict(xs=HALF), dict(w=None), dict(w=EIGHT), dict(ldw=24),
               dict(ldw=40), dict(ws=None), dict(y=None), dict(y=ODD), dict(y=HALF, dtype=0), dict(ldy=7), dict(offsets=HALF),
               dict(offsets=FAKE, order=FAKE, topk=0), dict(offsets=FAKE, order=HALF)):
        assert f(**kw) == BAD, kw
    for kw in (dict(k=40, ldx=48, ldw=48), dict(dtype=9), dict(offsets=FAKE, E=1025), dict(M=(1 << 26) + 1, rows=1 << 27),
               dict(n=(1 << 22) + 1, ldy=1 << 23), dict(k=(1 << 22) + 16, ldx=1 << 23, ldw=1 << 23), dict(ldx=1 << 23), dict(ldw=1 << 23),
               dict(offsets=FAKE, order=FAKE, rows=1 << 27), dict(M=1 << 26, rows=1 << 26, n=1 << 22, ldy=1 << 22)):
        assert f(**kw) == UNSUP, kw
    assert f(M=0, x=None, w=None, y=None, xs=None, ws=None) == OK


def _tensor(B, param=0x100000, grad=0x200000, copy=None, rows=3, cols=5, lp=5, lg=5, lc=0, dp=0, dg=1, dc=0):
    return B._AdamWTensor(param, grad, copy, rows, cols, lp, lg, lc, dp, dg, dc, 0)


def _pack(B, tensors, short=0):
    lib = B.load_library()
    n = len(tensors)
    items = (B._AdamWTensor * max(1, n))(*tensors)
    need = int(lib.logra_adamw_table_bytes(n))
    host = np.zeros(max(1, need // 8), np.uint64)
    desc = B._AdamWListDesc()
    st = lib.logra_adamw_list_pack(n, items, host.ctypes.data_as(ctypes.c_void_p), need - short, ctypes.byref(desc))
    return st, desc, host


def test_adamw_pack(B):
    st, desc, host = _pack(B, [_tensor(B), _tensor(B, None, None, rows=0), _tensor(B, 0x300000, 0x400000, 0x500000, 1, 700, 900, 800, 750, 1, 0, 1),
                               _tensor(B, 0x600000, 0x700000, rows=256, cols=1, lp=3, lg=1)])
    assert st == OK and desc.n == 4 and desc.blocks == 1 + 0 + 3 + 1 and desc.elements == 15 + 700 + 256
    e = host.reshape(4, -1)
    assert list(e[0][:10]) == [0x100000, 0x200000, 0, 3, 5, 5, 5, 0, 0, 1]
    assert list(e[2][:10]) == [0x300000, 0x400000, 0x500000, 1, 700, 700, 700, 700, 1, 3]       # one row: no stride
    assert list(e[3][:10]) == [0x600000, 0x700000, 0, 256, 1, 3, 1, 0, 4, 1]
    assert list(e[2][10:].view(np.int32)[:3]) == [1, 0, 1]
    st, desc, _ = _pack(B, [])
    assert st == OK and desc.blocks == 0


def test_adamw_pack_refusals(B):
    t = lambda **kw: _tensor(B, **kw)  # noqa: E731
    for bad in (t(rows=-1), t(cols=-1), t(lp=4), t(lg=4), t(copy=0x300000, lc=4), t(param=None), t(grad=None), t(param=0x100002),
                t(grad=0x200001), t(copy=0x300001, lc=5, dc=1), t(param=0x200000), t(copy=0x100010, lc=5), t(copy=0x200004, lc=5)):
        assert _pack(B, [bad])[0] == BAD
    assert _pack(B, [t(), t(grad=0x300000)])[0] == BAD                                    # one parameter twice
    assert _pack(B, [t(), t(param=0x400000)])[0] == BAD                                   # one gradient twice
    for bad in (t(dp=2), t(dg=7), t(dc=-1), t(rows=BIG, cols=2, lp=2, lg=2), t(lp=BIG)):
        assert _pack(B, [bad])[0] == UNSUP
    assert _pack(B, [t()], short=8)[0] == WS
    lib = B.load_library()
    assert lib.logra_adamw_table_bytes(-1) == 0 and lib.logra_adamw_table_bytes((1 << 20) + 1) == 0
    assert lib.logra_adamw_list_pack(1, None, FAKE, 1 << 20, ctypes.byref(B._AdamWListDesc())) == BAD


def test_adamw_refusals(B):
    lib = B.load_library()
    _, desc, _ = _pack(B, [_tensor(B)])
    desc.table = 0x900000
    none = B._AdamWListDesc()
    odd = B._AdamWListDesc(0x900008, 15, 1, 1, 0)
    f = _with(lib.logra_adamw, dict(list=ctypes.byref(desc), bits=8, m=FAKE, v=FAKE2, s=FAKE3, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8,
                                    wd=0.1, step=1, norm=None, most=1.0, seed=0, stream=None))
    nan, inf = float("nan"), float("inf")
    for kw in (dict(list=None), dict(list=ctypes.byref(odd)), dict(m=None), dict(v=None), dict(m=EIGHT), dict(v=EIGHT), dict(v=FAKE),
               dict(s=None), dict(s=HALF), dict(lr=nan), dict(lr=inf), dict(b1=1.0), dict(b1=-0.1), dict(b1=nan), dict(b2=1.0),
               dict(b2=nan), dict(eps=-1e-9), dict(eps=1e-40), dict(eps=nan), dict(eps=inf), dict(wd=nan), dict(step=0), dict(norm=HALF),
               dict(most=-1.0), dict(most=nan)):
        assert f(**kw) == BAD, kw
    assert f(bits=16) == UNSUP
    assert f(list=ctypes.byref(none), m=None, v=None, s=None) == OK


def test_binding_refuses_before_the_library(B):
    """Shapes and types that the binding looks at itself (on CPU tensors, which it refuses last)."""
    import rank_gradient_sketching_sketch_amd as L
    x, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for args, kw in (((x[0], ids, w), {}), ((x, ids.long(), w), {}), ((x, ids[:3], w), {}), ((x, ids, w[:, :1]), {}),
                     ((x, ids, w.double()), {}), ((x, ids, w), dict(bias=torch.zeros(7))), ((x.t(), ids, w), {}), ((x, ids, w), {}),
                     ((x, ids.t().contiguous().t(), w), {})):
        with pytest.raises(L.LograError):
            L.logra_route(*args, **kw)
    for args in ((x, ids, w, x[:, :7]), (x, ids, w, x.bfloat16()), (x, ids, w, x[:3]), (x, ids, w[:, :1], x), (x, ids, w, x)):
        with pytest.raises(L.LograError):
            L.logra_route_backward(*args)
    f8 = torch.float8_e4m3fn
    c, s = torch.zeros(4, 160, dtype=f8), torch.zeros(4, 2)
    x = torch.zeros(4, 160)
    for args, kw in (((x, c[:, :128], s), {}), ((x, c, s[:, :1]), {}), ((x, c.view(torch.uint8), s), {}), ((x, c, s), dict(block_rows=64)),
                     ((x, c, s), dict(block_rows=128)), ((x, c, torch.zeros(1, 2)), dict(block_rows=128, transpose=True)), ((x, c[None], s), {}),
                     ((x[:, ::2], c[:, :80], s), {}), ((x, c, s), {}), ((x.half(), c, s), {}),
                     ((torch.zeros(3, 4, 160)[:, :3], torch.zeros(3, 3, 160, dtype=f8), torch.zeros(3, 3, 2)), {})):
        with pytest.raises(L.LograError):
            L.logra_fp8_quantize(*args, **kw)
    w, ws, y = torch.zeros(16, 160, dtype=f8), torch.zeros(1, 2), torch.zeros(4, 16)
    off = torch.zeros(3, dtype=torch.int32)
    for args, kw in (((c, s, w[:, :128], ws, y), {}), ((c, s[:, :1], w, ws, y), {}), ((c, s, w, ws.t(), y), {}), ((c, s, w, ws, y[:, :15]), {}),
                     ((c, s, w, ws, y), dict(offsets=off)), ((c, s, torch.stack([w, w]), ws, y), dict(offsets=off)),
                     ((c, s, torch.stack([w, w]), torch.stack([ws, ws]), y), {}), ((c, s, w, ws, y), {}), ((x, s, w, ws, y), {}),
                     ((c, s, torch.stack([w, w]), torch.stack([ws, ws]), y), dict(offsets=off.long())),
                     ((c, s, torch.stack([w, w]), torch.stack([ws, ws]), y), dict(offsets=off, order=off))):
        with pytest.raises(L.LograError):
            L.logra_fp8_matmul(*args, **kw)
    p = torch.zeros(8)
    for args, kw in ((([p], []), {}), (([p], [p]), {}), (([p], [torch.zeros(8)]), dict(state_bits=16)), (([], []), dict(device="cpu"))):
        with pytest.raises(L.LograError):
            L.AdamWList(*args, **kw)
