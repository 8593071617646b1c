"""Host-side checks of gradient clipping and the expert-layer calls: the
packed table, every refusal (each returns before any launch), and the
oracle's own consistency. No GPU."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from oracle import experts as ox

FAKE, FAKE2 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10001)
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


def _pack(B, tensors, table_bytes=None):
    """tensors: (data, rows, cols, ld, dtype). Returns (status, desc, table)."""
    lib = B.load_library()
    n = len(tensors)
    items = (B._GradTensor * max(1, n))(*[B._GradTensor(*t, 0) for t in tensors])
    need = int(lib.logra_grad_table_bytes(n))
    host = np.zeros(max(1, need // 8), dtype=np.uint64)
    desc = B._GradListDesc()
    st = lib.logra_grad_list_pack(n, items, host.ctypes.data_as(ctypes.c_void_p),
                                  need if table_bytes is None else table_bytes, ctypes.byref(desc))
    return st, desc, host


def _entry(host, i, n):
    """(addr, rows, cols, ld, first, chunks, rows_per_chunk, segs_per_row, seg_len, bf16)"""
    e = host.reshape(n, -1)[i]
    tail = e[6:].view(np.int32)
    return tuple(int(x) for x in e[:6]) + tuple(int(x) for x in tail)


def test_pack_cuts_every_tensor_whole(B):
    shapes = [(0x100000, 3, 5, 5, 0), (0x200000, 1, 8192, 8192, 1), (0x300000, 1, 8193, 8193, 0),
              (0x400000, 4, 50001, 60000, 1), (None, 0, 7, 7, 0), (0x800000, 20000, 1, 3, 0), (0x900000, 7, 100, 100, 0)]
    st, desc, host = _pack(B, shapes)
    assert st == OK and desc.n == len(shapes)
    assert desc.elements == sum(r * c for _, r, c, _, _ in shapes)
    first = 0
    for i, (addr, r, c, ld, dt) in enumerate(shapes):
        a, rows, cols, eld, f, chunks, rpc, spr, seg, bf = _entry(host, i, len(shapes))
        assert (a, rows, cols, bf, f) == (addr or 0, r, c, dt, first)
        covered = np.zeros((r, c), np.int8)
        for k in range(chunks):
            if rpc > 0:
                assert rpc * c <= 8192
                covered[k * rpc:(k + 1) * rpc] += 1
                assert k * rpc < r
            else:
                row, s = divmod(k, spr)
                assert 0 < seg <= 8192 and s * seg < c
                covered[row, s * seg:(s + 1) * seg] += 1
        assert (covered == 1).all()
        first += chunks
    assert desc.chunks == first
    # the cut and the shapes' hash depend on rows and cols alone
    st, other, _ = _pack(B, [(0x10000000 + (a or 0), r, c, c, 1 - dt) for a, r, c, ld, dt in shapes if a] )
    st2, same, _ = _pack(B, [(0x20000000 + 4 * (a or 0), r, c, c + 9, dt) for a, r, c, ld, dt in shapes if a])
    assert st == OK and st2 == OK and (other.shapes, other.chunks) == (same.shapes, same.chunks)
    st, swapped, _ = _pack(B, [(0x100000, 5, 3, 3, 0)])
    st, plain, _ = _pack(B, [(0x100000, 3, 5, 5, 0)])
    assert swapped.shapes != plain.shapes


def test_pack_refusals(B):
    good = (0x100000, 3, 5, 5, 0)
    assert _pack(B, [good])[0] == OK
    assert _pack(B, [])[0] == OK
    assert _pack(B, [(0x100000, -1, 5, 5, 0)])[0] == BAD
    assert _pack(B, [(0x100000, 3, -5, 5, 0)])[0] == BAD
    assert _pack(B, [(0x100000, 3, 5, 4, 0)])[0] == BAD
    assert _pack(B, [(0x100002, 3, 5, 5, 0)])[0] == BAD          # fp32 off its alignment
    assert _pack(B, [(0x100002, 3, 5, 5, 1)])[0] == OK
    assert _pack(B, [(0x100001, 3, 5, 5, 1)])[0] == BAD
    assert _pack(B, [(None, 3, 5, 5, 0)])[0] == BAD
    assert _pack(B, [(None, 3, 0, 0, 0)])[0] == OK
    assert _pack(B, [(0x100000, 3, 5, 5, 2)])[0] == UNSUP
    assert _pack(B, [(0x100000, 1 << 30, 1 << 30, 1 << 30, 0)])[0] == UNSUP
    assert _pack(B, [good], table_bytes=8)[0] == WS
    # the same tensor twice, overlaps, interleaved views; neighbours are fine
    assert _pack(B, [good, good])[0] == BAD
    assert _pack(B, [good, (0x100000 + 56, 1, 5, 5, 0)])[0] == BAD
    assert _pack(B, [(0x100000 + 60, 1, 5, 5, 0), good])[0] == OK
    assert _pack(B, [(0x100000, 4, 8, 16, 0), (0x100000 + 32, 4, 8, 16, 0)])[0] == BAD
    lib = B.load_library()
    d = B._GradListDesc()
    assert lib.logra_grad_list_pack(-1, None, None, 0, ctypes.byref(d)) == BAD
    assert lib.logra_grad_list_pack(1, None, FAKE, 1 << 20, ctypes.byref(d)) == BAD
    assert lib.logra_grad_list_pack((1 << 20) + 1, None, FAKE, BIG, ctypes.byref(d)) == BAD
    assert lib.logra_grad_table_bytes(-1) == 0


def test_clip_refusals(B):
    lib = B.load_library()
    r = ctypes.byref
    _, d, _ = _pack(B, [(0x100000, 300, 256, 256, 0)])
    _, o, _ = _pack(B, [(0x900000, 300, 256, 256, 1)])
    _, other, _ = _pack(B, [(0x900000, 256, 300, 300, 1)])
    need = B.load_library().logra_grad_workspace_bytes(r(d))
    assert 0 < need <= 2048 * 8

    def clip(lst=d, out=None, mx=1.0, norm=FAKE, coef=FAKE2, ws=FAKE, wsb=need):
        return lib.logra_grad_clip(None if lst is None else r(lst), None if out is None else r(out), ctypes.c_float(mx),
                                   norm, coef, ws, wsb, None)

    assert clip() == BAD                                # the table has no device address yet
    d.table = o.table = other.table = 0x40000
    assert clip(lst=None) == BAD
    assert clip(mx=-1.0) == BAD and clip(mx=float("nan")) == BAD
    assert clip(norm=None) == BAD and clip(coef=None) == BAD and clip(coef=FAKE) == BAD and clip(norm=ODD) == BAD
    assert clip(out=other) == BAD                       # other shapes
    assert clip(ws=None) == WS and clip(wsb=need - 8) == WS and clip(ws=ctypes.c_void_p(0x10008)) == WS
    d.table = 0x40008
    assert clip() == BAD
    d.table = 0x40000
    assert lib.logra_grad_norm(r(d), None, FAKE, need, None) == BAD
    assert lib.logra_grad_norm(r(d), FAKE2, FAKE, 0, None) == WS
    assert lib.logra_grad_norm(None, FAKE2, FAKE, need, None) == BAD
    assert lib.logra_grad_workspace_bytes(None) == 0
    # few elements in few tensors are done by one workgroup, without a workspace
    for shapes, few in (([(1, 32768)], True), ([(1, 32769)], False), ([(1, 8)] * 32, True), ([(1, 8)] * 33, False)):
        _, s, _ = _pack(B, [(0x100000 * (i + 1), n, c, c, 0) for i, (n, c) in enumerate(shapes)])
        assert (lib.logra_grad_workspace_bytes(r(s)) == 0) == few


def test_expert_refusals(B):
    lib = B.load_library()

    def sort(T=4, K=2, E=8, ids=FAKE, nb=4, ld=2, off=FAKE, order=FAKE, slots=FAKE, ws=None, wsb=0):
        return lib.logra_expert_sort(T, K, E, ids, nb, ld, off, order, slots, ws, wsb, None)

    assert sort(T=-1) == BAD and sort(K=0) == BAD and sort(E=0) == BAD and sort(ids=None) == BAD and sort(nb=2) == BAD
    assert sort(ld=1) == BAD and sort(off=None) == BAD and sort(order=None) == BAD and sort(slots=None) == BAD
    assert sort(ids=ctypes.c_void_p(0x10004), nb=8) == BAD and sort(slots=ODD) == BAD
    assert sort(K=65, ld=65) == UNSUP and sort(E=1025) == UNSUP and sort(T=(1 << 23) + 1) == UNSUP
    assert sort(T=1 << 23, K=16, ld=16) == UNSUP
    need = lib.logra_expert_sort_workspace_bytes(9000, 2, 8)
    assert need > 0 and lib.logra_expert_sort_workspace_bytes(4, 2, 8) == 0
    assert sort(T=9000) == WS and sort(T=9000, ws=FAKE, wsb=need - 1) == WS
    assert lib.logra_expert_sort_workspace_bytes(-1, 2, 8) == 0 and lib.logra_expert_sort_workspace_bytes(4, 2, 0) == 0

    def gather(T=4, K=2, h=16, dt=1, X=FAKE, ldx=16, slots=FAKE, w=None, Xs=FAKE2, ldxs=16, n=8):
        return lib.logra_expert_gather(T, K, h, dt, X, ldx, slots, w, Xs, ldxs, n, None)

    def combine(T=4, K=2, h=16, dt=1, Ys=FAKE, ldys=16, n=8, slots=FAKE, w=None, Y=FAKE2, ldy=16):
        return lib.logra_expert_combine(T, K, h, dt, Ys, ldys, n, slots, w, Y, ldy, None)

    def back(T=4, K=2, h=16, dt=1, dY=FAKE, ldd=16, Ys=FAKE, ldys=16, n=8, slots=FAKE, w=FAKE, dYs=FAKE2, lds=16, dw=FAKE2):
        return lib.logra_expert_combine_backward(T, K, h, dt, dY, ldd, Ys, ldys, n, slots, w, dYs, lds, dw, None)

    for f in (gather, combine, back):
        assert f(T=-1) == BAD and f(K=0) == BAD and f(h=0) == BAD and f(n=-1) == BAD and f(slots=None) == BAD
        assert f(dt=2) == UNSUP and f(K=65) == UNSUP and f(T=(1 << 23) + 1) == UNSUP and f(w=ODD) == BAD
        assert f(h=1 << 31) == UNSUP
        assert f(T=0, slots=None) == OK                # nothing to do, nothing launched
    assert gather(X=None) == BAD and gather(Xs=None) == BAD and gather(ldx=15) == BAD and gather(ldxs=15) == BAD
    assert gather(X=ODD) == BAD and gather(Xs=ctypes.c_void_p(0x20002), dt=0) == BAD
    assert gather(n=0, Xs=None) == OK
    assert combine(Ys=None) == BAD and combine(Y=None) == BAD and combine(ldys=15) == BAD and combine(ldy=1) == BAD
    assert back(w=None) == BAD and back(dw=None) == BAD and back(dY=None) == BAD and back(Ys=None) == BAD
    assert back(dYs=None) == BAD and back(lds=3) == BAD


def test_sketch_experts_refusals(B):
    lib = B.load_library()
    m = B.MatrixDesc(64, 128, 32)
    need = B.logra_sketch_experts_workspace_bytes(m, 4, 100, 1)
    assert need > 0

    def call(m=m, E=4, N=100, dt=1, off=FAKE, order=FAKE, K=2, X=FAKE, ldx=128, rows=50, dY=FAKE, ldd=64, S=FAKE2, acc=0,
             ws=FAKE, wsb=need):
        return lib.logra_sketch_experts(None if m is None else ctypes.byref(m), E, 1, N, dt, off, order, K, X, ldx, rows,
                                        dY, ldd, S, acc, ws, wsb, None)

    assert call(m=None) == BAD and call(E=0) == BAD and call(N=-1) == BAD and call(off=None) == BAD and call(S=None) == BAD
    assert call(K=0) == BAD and call(order=None, rows=99) == BAD and call(rows=-1) == BAD
    assert call(X=None) == BAD and call(dY=None) == BAD and call(ldx=120) == BAD and call(ldd=56) == BAD
    assert call(ldx=132) == BAD and call(ldd=68) == BAD and call(X=ctypes.c_void_p(0x10008)) == BAD
    assert call(S=ctypes.c_void_p(0x20008)) == BAD and call(off=ODD) == BAD
    assert call(E=1025) == UNSUP and call(N=(1 << 26) + 1) == UNSUP and call(dt=5) == UNSUP
    assert call(m=B.MatrixDesc(64, 128, 48)) == UNSUP and call(m=B.MatrixDesc(60, 128, 32)) == UNSUP
    assert call(m=B.MatrixDesc(64, 128, 2000), dt=0) == UNSUP
    assert call(m=B.MatrixDesc((1 << 22) + 8, 128, 32), ldd=1 << 23) == UNSUP
    assert call(m=B.MatrixDesc(64, (1 << 22) + 8, 32), ldx=1 << 23) == UNSUP
    assert call(E=1024, m=B.MatrixDesc(1 << 22, 128, 32), ldd=1 << 22) == UNSUP     # S past one launch
    assert call(ldx=1 << 25, rows=32) == UNSUP                  # X past one buffer view (2^31 bytes)
    assert call(ldx=(1 << 25) - 8, rows=32, wsb=0) == WS
    assert call(ldd=(1 << 24) + 8) == UNSUP
    assert call(ws=None) == WS and call(wsb=need - 1) == WS and call(ws=ctypes.c_void_p(0x10008)) == WS
    assert call(N=0, acc=1, ws=None, wsb=0, X=None, dY=None) == OK
    assert B.logra_sketch_experts_workspace_bytes(B.MatrixDesc(64, 128, 48), 4, 100, 1) == 0
    assert B.logra_sketch_experts_workspace_bytes(m, 0, 100, 1) == 0


def test_binding_refuses_what_it_cannot_pass(B):
    ids = torch.zeros(4, 2, dtype=torch.int32)
    off, order, slots = (torch.zeros(n, dtype=torch.int32) for n in (9, 8, 8))
    X = torch.zeros(4, 16)
    with pytest.raises(B.LograError):                   # host tensors
        B.logra_expert_sort(ids, 8, off, order, slots.view(4, 2))
    with pytest.raises(B.LograError):
        B.logra_expert_sort(ids.float(), 8, off, order, slots.view(4, 2))
    with pytest.raises(B.LograError):
        B.logra_expert_sort(ids, 7, off, order, slots.view(4, 2))
    with pytest.raises(B.LograError):
        B.logra_expert_gather(X, slots.view(4, 2), torch.zeros(8, 15))
    with pytest.raises(B.LograError):
        B.logra_expert_gather(X, slots.view(4, 2), torch.zeros(8, 16, dtype=torch.bfloat16))
    with pytest.raises(B.LograError):
        B.logra_expert_gather(X.t(), slots.view(4, 2), torch.zeros(8, 16))
    with pytest.raises(B.LograError):
        B.logra_expert_gather(X, slots.view(2, 4), torch.zeros(8, 16))
    with pytest.raises(B.LograError):
        B.logra_expert_combine(torch.zeros(8, 16), slots.view(4, 2), X, weights=torch.zeros(4, 3))
    with pytest.raises(B.LograError):
        B.logra_expert_combine(torch.zeros(8, 16).half(), slots.view(4, 2), X.half())
    with pytest.raises(B.LograError):
        B.logra_expert_combine_backward(X, torch.zeros(8, 16), slots.view(4, 2), torch.zeros(4, 2), torch.zeros(7, 16),
                                        torch.zeros(4, 2))
    with pytest.raises(B.LograError):
        B.GradList([torch.zeros(3)])
    with pytest.raises(B.LograError):
        B.logra_sketch_experts(B.MatrixDesc(16, 16, 32), off, torch.zeros(8, 16), torch.zeros(8, 16),
                               torch.zeros(8, 16, 16), False)


def test_oracle_agrees_with_matrix_forms():
    g = np.random.default_rng(0)
    T, K, E, h = 30, 3, 5, 7
    ids = g.integers(-1, E + 1, (T, K))
    offsets, order, slots = ox.expert_sort(ids, E)
    kept = offsets[-1]
    # a permutation matrix of the kept pairs says the same
    perm = np.zeros((T * K, T * K))
    flat = slots.reshape(-1)
    perm[flat[flat >= 0], np.nonzero(flat >= 0)[0]] = 1
    assert (np.sort(order[:kept]) == np.nonzero(flat >= 0)[0]).all() and (order[kept:] == -1).all()
    e = ids.reshape(-1)[order[:kept]]
    assert (np.diff(e) >= 0).all() and all((np.diff(order[:kept][e == x]) > 0).all() for x in range(E))
    X, w = g.standard_normal((T, h)), g.standard_normal((T, K))
    spread = np.kron(np.eye(T), np.ones((K, 1)))        # token -> its pairs
    D = perm @ (w.reshape(-1, 1) * spread)
    assert np.allclose(ox.gather(X, slots, w, np.zeros((T * K, h))), D @ X)
    Ys, dY = g.standard_normal((T * K, h)), g.standard_normal((T, h))
    assert np.allclose(ox.combine(Ys, slots, w)[0], D.T @ Ys)
    dYs, dw, _ = ox.combine_backward(dY, Ys, slots, w, np.zeros((T * K, h)))
    assert np.allclose(dYs, D @ dY)
    full = np.einsum("th,tjh->tj", dY, (perm.T @ Ys).reshape(T, K, h))
    assert np.allclose(dw, full)
    norm, coef, out = ox.clip([X, w], 1.0)
    assert math.isclose(np.sqrt(sum((o ** 2).sum() for o in out)), 1.0) and math.isclose(coef * norm, 1.0)
    S, _, _ = ox.sketch_experts(X[np.clip(order // K, 0, T - 1)], Ys, offsets, h, h, 16, 0, 1, 2, 3)
    from oracle import sign_matrix
    a, b = offsets[1], offsets[2]
    G = Ys[a:b].T @ X[order[a:b] // K]
    assert np.allclose(S[1], G @ sign_matrix(0, 1, 5, 16, h).T)
