"""The sketch over experts against the plain fp64 oracle.

Tolerances. bf16: per entry, P's three-term form is off by at most 2^-24 |P|
(each bf16 rounding is 2^-8 of what it rounds), its fp32 accumulation by
(k + 16) 2^-23 of c sum |X| and that of S by (3 n + 16) 2^-23 of
sum |dY| |P| (2^-23: the matrix cores' additions are not taken to round to
nearest). Over all entries those errors are independent: the accumulations'
root mean square is below sqrt(k + 3 n) 2^-23, so the relative Frobenius error
stays below 1e-5. fp32:
(k + n + 8) 2^-23 of the magnitudes, and 1e-5 likewise."""
import numpy as np
import pytest
import torch

import oracle
import rank_gradient_sketching_sketch_amd as L
from rank_gradient_sketching_sketch_amd import binding as B
from oracle import experts as ox
from gpu_util import device, say

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().cpu().double().numpy()


def _inputs(seed, T, K, E, d, k, dt, dev, drop=0.1, popular=None, pad=0):
    g = np.random.default_rng(seed)
    ids = g.integers(0, E, (T, K)) if popular is None else np.full((T, K), popular)
    ids = np.where(g.random((T, K)) < drop, -1, ids)
    offsets, order, slots = (torch.from_numpy(x).to(dev) for x in ox.expert_sort(ids, E))
    tg = torch.Generator().manual_seed(seed)
    X = torch.randn(T, k + pad, generator=tg).to(dt).to(dev)[:, :k]
    dY = (torch.randn(T * K, d + pad, generator=tg) * 1e-3).to(dt).to(dev)[:, :d]
    return offsets, order, X, dY


def _check(S, ref, mag_p, mag_x, k, n, bf16):
    S = _f64(S)
    u = 2.0 ** -23
    if bf16:
        bound = (2.0 ** -24 + (3 * n + 16) * u) * mag_p + (k + 16) * u * (1 + 2.0 ** -8) * mag_x
    else:
        bound = (k + n + 8) * u * (mag_x + mag_p)
    assert np.all(np.abs(S - ref) <= bound + 1e-30)
    size = np.linalg.norm(ref)
    if size:
        assert np.linalg.norm(S - ref) <= 1e-5 * size


CASES = [
    # T, K, E, d, k, r, popular expert, pad of the rows
    (1, 1, 1, 8, 8, 32, None, 0),
    (1, 8, 128, 64, 72, 32, None, 0),
    (64, 2, 16, 256, 1536, 64, None, 0),
    (100, 3, 5, 200, 520, 256, None, 8),
    (33, 1, 2, 72, 64, 128, None, 16),
    (700, 4, 8, 136, 136, 256, None, 0),
    (400, 8, 8, 96, 64, 64, 3, 0),         # one expert holds every row: its rows are split over items
    (1500, 4, 16, 264, 40, 32, 15, 8),
    (31, 2, 70, 40, 2056, 256, None, 0),   # more experts than a wave has lanes
    (900, 2, 3, 1000, 200, 128, None, 0),
    # enough rows for the wide projection: ragged k, padded rows, one popular expert, more experts than lanes
    (1100, 4, 9, 136, 520, 256, None, 8),
    (2100, 2, 5, 72, 200, 128, None, 0),
    (1200, 4, 70, 40, 2056, 256, 3, 0),
    (4100, 1, 3, 64, 72, 128, None, 16),
    (600, 8, 130, 64, 128, 256, None, 0),
    # 64 columns per workgroup of the other projection, of 256 and of 64
    (900, 2, 4, 72, 712, 256, 2, 8),
    (3001, 2, 6, 64, 72, 64, None, 0),
    # the most experts
    (1500, 2, 1024, 16, 72, 256, None, 0),
    (700, 1, 1024, 8, 64, 32, None, 0),
    (6000, 1, 1024, 8, 64, 128, 1023, 0),
]


@pytest.mark.parametrize("T,K,E,d,k,r,popular,pad", CASES)
def test_bf16_matches_oracle(T, K, E, d, k, r, popular, pad):
    dev = device()
    say("sketch experts bf16", T, K, E, d, k, r, popular, pad)
    offsets, order, X, dY = _inputs(T + d, T, K, E, d, k, torch.bfloat16, dev, popular=popular, pad=pad)
    m = L.MatrixDesc(d, k, r, seed=5, step=2, matrix_id=40)
    S = torch.full((E, d, r), float("nan"), device=dev)
    L.logra_sketch_experts(m, offsets, X, dY, S, False, order=order, topk=K, id_stride=7)
    o = offsets.cpu().numpy()
    ref, mp, mx = ox.sketch_experts(_f64(X), _f64(dY), o, d, k, r, 5, 2, 40, 7, order=order.cpu().numpy(), topk=K)
    n = int(np.diff(o).max())
    _check(S, ref, mp, mx, k, n, True)
    # a second microbatch on top, from the sorted copy of X: the same rows again
    Xs = torch.zeros(T * K, k, dtype=X.dtype, device=dev)
    Xs[:o[-1]] = X[order[:o[-1]].long() // K]
    L.logra_sketch_experts(m, offsets, Xs, dY, S, True, id_stride=7)
    _check(S, 2 * ref, 2 * mp, 2 * mx, k, n, True)


@pytest.mark.parametrize("T,K,E,d,k,r,popular,pad", [(1, 1, 1, 3, 5, 1, None, 0), (40, 2, 6, 45, 130, 20, None, 3),
                                                     (384, 2, 8, 256, 512, 32, None, 0), (50, 4, 70, 33, 64, 40, 2, 0),
                                                     (200, 2, 70, 260, 97, 100, None, 5)])
def test_f32_matches_oracle(T, K, E, d, k, r, popular, pad):
    dev = device()
    say("sketch experts f32", T, K, E, d, k, r, popular, pad)
    offsets, order, X, dY = _inputs(T + d, T, K, E, d, k, torch.float32, dev, popular=popular, pad=pad)
    m = L.MatrixDesc(d, k, r, seed=1, step=9, matrix_id=3)
    S = torch.full((E, d, r), float("nan"), device=dev)
    L.logra_sketch_experts(m, offsets, X, dY, S, False, order=order, topk=K)
    o = offsets.cpu().numpy()
    ref, mp, mx = ox.sketch_experts(_f64(X), _f64(dY), o, d, k, r, 1, 9, 3, 1, order=order.cpu().numpy(), topk=K)
    _check(S, ref, mp, mx, k, int(np.diff(o).max()), False)
    L.logra_sketch_experts(m, offsets, X, dY, S, True, order=order, topk=K)
    _check(S, 2 * ref, 2 * mp, 2 * mx, k, int(np.diff(o).max()), False)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_no_rows_at_all(dt):
    dev = device()
    E, d, k, r = 6, 72, 40, 32
    m = L.MatrixDesc(d, k, r)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    S = torch.full((E, d, r), 3.0, device=dev)
    for T in (0, 10):                       # no tokens; tokens that no expert holds
        X, dY = torch.randn(T, k, device=dev).to(dt), torch.full((T, d), float("nan"), device=dev).to(dt)
        S.fill_(3.0)
        L.logra_sketch_experts(m, offsets, X, dY, S, True)
        assert (S == 3.0).all()
        L.logra_sketch_experts(m, offsets, X, dY, S, False)
        assert not S.any()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_and_tokens_that_are_not_named_are_not_read(dt):
    """NaN in dY behind the last sorted row and in X rows that no kept pair
    names changes nothing; an order entry outside X counts as zeros; offsets
    beyond the rows are cut."""
    dev = device()
    T, K, E, d, k, r = 45, 2, 4, 64, 72, 32
    offsets, order, X, dY = _inputs(1, T, K, E, d, k, dt, dev, drop=0.5)
    m = L.MatrixDesc(d, k, r, matrix_id=1)
    kept = int(offsets[-1])
    S, S2 = torch.empty(E, d, r, device=dev), torch.empty(E, d, r, device=dev)
    L.logra_sketch_experts(m, offsets, X, dY, S, False, order=order, topk=K)
    used = torch.zeros(T, dtype=torch.bool, device=dev)
    used[order[:kept].long() // K] = True
    X2, dY2 = X.clone(), dY.clone()
    assert not used.all() and kept < T * K
    X2[~used] = float("nan")
    dY2[kept:] = float("nan")
    L.logra_sketch_experts(m, offsets, X2, dY2, S2, False, order=order, topk=K)
    assert torch.equal(S, S2)
    far = order.clone()
    far[0], far[1] = -1, T * K + 5
    L.logra_sketch_experts(m, offsets, X2, dY2, S2, False, order=far, topk=K)
    dY3 = dY.clone()
    dY3[:2] = 0
    L.logra_sketch_experts(m, offsets, X, dY3, S, False, order=order, topk=K)
    assert torch.allclose(S, S2, rtol=1e-4, atol=1e-7)
    cut = offsets.clone()
    cut[-1] = 1 << 30
    cut[0] = -5
    full = offsets.clone()
    full[-1] = T * K
    full[0] = 0
    order_full = order.clamp(min=0)
    L.logra_sketch_experts(m, cut, X, dY, S, False, order=order_full, topk=K)
    L.logra_sketch_experts(m, full, X, dY, S2, False, order=order_full, topk=K)
    assert torch.equal(S, S2)


@pytest.mark.parametrize("T,r,dt", [(60, 64, torch.bfloat16), (2500, 256, torch.bfloat16), (60, 32, torch.float32)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_reach_their_own_expert_only(T, r, dt, bad):
    """A token's non-finite activation or output gradient makes the sketches
    of its experts non-finite and no other's (T = 2500: the wide projection)."""
    dev = device()
    K, E, d, k = 2, 6, 72, 136
    offsets, order, X, dY = _inputs(3, T, K, E, d, k, dt, dev, drop=0.3)
    m = L.MatrixDesc(d, k, r)
    o = offsets.tolist()
    S = torch.empty(E, d, r, device=dev)
    first = o[2] + 1                                          # a row of expert 2
    token = int(order[first]) // K
    held = {e for e in range(E) if any(int(p) // K == token for p in order[o[e]:o[e + 1]])}
    X2 = X.clone()
    X2[token, 5] = bad
    L.logra_sketch_experts(m, offsets, X2, dY, S, False, order=order, topk=K)
    for e in range(E):
        assert bool(torch.isfinite(S[e]).all()) == (e not in held)
    dY2 = dY.clone()
    dY2[first, 7] = bad
    L.logra_sketch_experts(m, offsets, X, dY2, S, False, order=order, topk=K)
    for e in range(E):
        assert bool(torch.isfinite(S[e]).all()) == (e != 2)
    assert not torch.isfinite(S[2, 7]).any() and torch.isfinite(S[2, :7]).all() and torch.isfinite(S[2, 8:]).all()


def test_same_as_the_one_matrix_sketch():
    """One expert with every row: the one-matrix call's S to the bf16 path's
    tolerance (that call rounds P to one bf16 term)."""
    dev = device()
    T, d, k, r = 300, 264, 520, 256
    offsets, order, X, dY = _inputs(2, T, 1, 1, d, k, torch.bfloat16, dev, drop=0)
    m = L.MatrixDesc(d, k, r, seed=4, step=1, matrix_id=6)
    S, S1 = torch.empty(1, d, r, device=dev), torch.empty(d, r, device=dev)
    L.logra_sketch_experts(m, offsets, X, dY, S, False)
    L.logra_sketch_accumulate(m, X.contiguous(), dY.contiguous(), S1, False)
    assert float((S[0] - S1).norm() / S1.norm()) < 2.0 ** -8


def test_rows_past_32_bit_offsets():
    dev = device()
    E, d, k, r, n = 4, 8200, 64, 32, 70000             # dY: 280000 rows of 16400 bytes, 4.6 GB
    g = torch.Generator(device=dev).manual_seed(3)
    N = E * n
    X = torch.randn(N, k, generator=g, device=dev).to(torch.bfloat16)
    dY = torch.zeros(N, d, dtype=torch.bfloat16, device=dev)
    live = torch.arange(n - 40, n, device=dev) + (E - 1) * n       # the last rows of all
    dY[live] = torch.randn(40, d, generator=g, device=dev).to(torch.bfloat16)
    offsets = torch.arange(0, N + 1, n, dtype=torch.int32, device=dev)
    m = L.MatrixDesc(d, k, r, matrix_id=11)
    S = torch.empty(E, d, r, device=dev)
    L.logra_sketch_experts(m, offsets, X, dY, S, False)
    ref, _, _ = ox.sketch_experts(_f64(X[live]), _f64(dY[live]), [0, 40], d, k, r, 0, 0, 11 + E - 1, 1)
    assert not S[:E - 1].any()
    assert np.linalg.norm(_f64(S[E - 1]) - ref[0]) <= 1e-5 * np.linalg.norm(ref[0])


def test_repeats_graph_and_side_stream():
    dev = device()
    T, K, E, d, k, r = 400, 8, 8, 96, 136, 64
    offsets, order, X, dY = _inputs(5, T, K, E, d, k, torch.bfloat16, dev, popular=2)
    m = L.MatrixDesc(d, k, r, step=4)
    ws = torch.empty(L.logra_sketch_experts_workspace_bytes(m, E, T * K, B.LOGRA_BF16), dtype=torch.uint8, device=dev)
    S = torch.empty(E, d, r, device=dev)

    def work(**kw):
        L.logra_sketch_experts(m, offsets, X, dY, S, False, order=order, topk=K, **kw)
        L.logra_sketch_experts(m, offsets, X, dY, S, True, order=order, topk=K, **kw)

    work(ws=ws)
    torch.cuda.synchronize()
    ref = S.clone()
    side = torch.cuda.Stream()
    for _ in range(2):
        S.zero_()
        side.wait_stream(torch.cuda.current_stream())
        work(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(S, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(ws=ws)
    for _ in range(3):
        work()
        S.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(S, ref)


def test_one_row_of_any_stride():
    """The row stride of a single row has no meaning: none is refused."""
    dev = device()
    offsets, order, X, dY = _inputs(12, 1, 1, 3, 40, 64, torch.bfloat16, dev)
    m = L.MatrixDesc(40, 64, 32, seed=1, step=0, matrix_id=0)
    want, got = torch.empty(3, 40, 32, device=dev), torch.empty(3, 40, 32, device=dev)
    L.logra_sketch_experts(m, offsets, X, dY, want, False, order=order, topk=1)
    for ld in (1, 67, 1 << 25):
        L.logra_sketch_experts(m, offsets, X.as_strided((1, 64), (ld, 1)), dY.as_strided((1, 40), (ld, 1)), got, False,
                               order=order, topk=1)
        assert torch.equal(want, got)


def test_f32_more_rows_than_one_row_of_the_grid():
    """2.24 million rows (70000 units of 32): whole numbers and halves, so
    that every sum is exact in fp32."""
    dev = device()
    N, E, d, r = 70000 * 32, 3, 2, 4
    g = torch.Generator().manual_seed(4)
    dY = torch.randint(0, 2, (N, d), generator=g).float().to(dev)
    X = torch.ones(N, 1, device=dev)
    bounds = [0, 1000003, 1000003, N - 5]
    offsets = torch.tensor(bounds, dtype=torch.int32, device=dev)
    S = torch.empty(E, d, r, device=dev)
    m = L.MatrixDesc(d, 1, r, seed=3, step=1, matrix_id=9)
    L.logra_sketch_experts(m, offsets, X, dY, S, False)
    for e in range(E):
        A = oracle.sign_matrix(3, 1, 9 + e, r, 1)
        sums = _f64(dY[bounds[e]:bounds[e + 1]]).sum(0)
        assert np.array_equal(_f64(S[e]), sums[:, None] * A[:, 0][None, :])
