"""Sort by expert, gather, combine and combine's gradient against the plain
fp64 oracle.

Tolerances. The sort is whole numbers: equal. A gather without weights copies
bits; with weights it is one fp32 product (2^-24) and, in bf16, one rounding
(2^-8). combine adds K products in fp32: K 2^-24 of the sum of magnitudes,
then the rounding of the result. dw is a sum over h in which a product passes
through at most ceil(h / (256 V)) V + 10 roundings (V = 8 or 4 elements per
thread and pass, 6 + 4 more to add the threads up)."""
import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from oracle import experts as ox
from gpu_util import device, say

pytestmark = pytest.mark.gpu


def _ids(seed, T, K, E, drop=0.1, dtype=torch.int32):
    g = np.random.default_rng(seed)
    ids = g.integers(0, E, (T, K))
    bad = g.random((T, K)) < drop
    ids = np.where(bad, g.choice([-1, E, E + 5, -7], (T, K)), ids)
    return torch.from_numpy(ids).to(dtype)


def _sort(ids, E, dev, **kw):
    T, K = ids.shape
    out = (torch.full((E + 1,), -99, dtype=torch.int32, device=dev),
           torch.full((T * K,), -99, dtype=torch.int32, device=dev),
           torch.full((T, K), -99, dtype=torch.int32, device=dev))
    L.logra_expert_sort(ids, E, *out, **kw)
    return out


def _same_sort(got, ids, E):
    for a, b in zip(got, ox.expert_sort(ids.cpu().numpy(), E)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("T,K,E", [(0, 2, 4), (1, 1, 1), (1, 8, 128), (16, 8, 128), (63, 1, 7), (65, 64, 3),
                                   (1000, 3, 60), (1024, 8, 8), (1025, 8, 256), (5000, 4, 1024), (300, 5, 1000),
                                   (30001, 2, 17), (512, 8, 64),
                                   (1366, 3, 1024), (70001, 8, 129)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, K, E, dtype):
    dev = device()
    say("sort", T, K, E, dtype)
    ids = _ids(T + K + E, T, K, E, dtype=dtype).to(dev)
    first = _sort(ids, E, dev)
    _same_sort(first, ids, E)
    wide = torch.full((T, K + 3), 1, dtype=dtype, device=dev)      # strided ids
    wide[:, 1:K + 1] = ids
    for a, b in zip(first, _sort(wide[:, 1:K + 1], E, dev)):
        assert torch.equal(a, b)


def test_sort_edges():
    dev = device()
    E = 16
    for ids in (torch.full((50, 4), -1), torch.full((3000, 4), 99), torch.full((70, 2), 5), torch.full((9000, 2), 15),
                torch.tensor([[3, 3, 3], [0, 3, 0]])):
        d = ids.to(torch.int32).to(dev)
        _same_sort(_sort(d, E, dev), d, E)
    # ids far outside 32 bits are dropped, not wrapped
    d = torch.tensor([[1 << 32, 2], [-(1 << 40), (1 << 33) + 2]], dtype=torch.int64, device=dev)
    _same_sort(_sort(d, E, dev), d, E)


def _case(seed, T, K, E, h, dt, dev, drop=0.1, pad=0, off=0):
    """Rows in wider buffers, `off` elements in: strides and odd alignment."""
    g = torch.Generator().manual_seed(seed)
    ids = _ids(seed, T, K, E, drop).to(dev)
    offsets, order, slots = _sort(ids, E, dev)
    n = T * K

    def rows(count, std=1.0):
        base = (torch.randn(count, h + pad, generator=g) * std).to(dt).to(dev)
        return base[:, off:off + h] if pad else base

    w = torch.rand(T, K, generator=g).to(dev)
    return dict(offsets=offsets, order=order, slots=slots, w=w, X=rows(T), Ys=rows(n), dY=rows(T), Xs=rows(n), dYs=rows(n),
                Y=rows(T))


def _f64(t):
    return t.detach().cpu().double().numpy()


ROWS = [(1, 1, 1, 1, 0, 0), (1, 8, 128, 2048, 0, 0), (5, 3, 4, 7, 3, 1), (33, 8, 16, 256, 8, 0), (40, 2, 8, 1499, 0, 0),
        (9, 6, 60, 1000, 5, 3), (17, 1, 3, 4100, 4, 4), (3, 64, 8, 520, 0, 0), (200, 4, 8, 64, 0, 0),
        (64, 9, 5, 9000, 2, 1), (6, 3, 4, 9, 2, 1), (12, 5, 6, 2049, 0, 0), (1200, 3, 5, 14001, 3, 1)]      # the last: more than 96 MB of rows


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E,h,pad,off", ROWS)
def test_rows_match_oracle(T, K, E, h, pad, off, dt):
    dev = device()
    say("rows", T, K, E, h, pad, off, dt)
    c = _case(T + h, T, K, E, h, dt, dev, pad=pad, off=off)
    slots, w = c["slots"].cpu().numpy(), _f64(c["w"])
    half = 2.0 ** -8 if dt == torch.bfloat16 else 0.0
    tiny = 1e-37
    # gather: copies, then weighted
    before = c["Xs"].clone()
    L.logra_expert_gather(c["X"], c["slots"], c["Xs"])
    assert np.array_equal(_f64(c["Xs"]), ox.gather(_f64(c["X"]), slots, None, _f64(before)))
    c["Xs"].copy_(before)
    L.logra_expert_gather(c["X"], c["slots"], c["Xs"], weights=c["w"])
    ref = ox.gather(_f64(c["X"]), slots, w, _f64(before))
    assert np.all(np.abs(_f64(c["Xs"]) - ref) <= (half + 2.0 ** -23) * np.abs(ref) + tiny)
    # combine, weighted and not
    for weights, wr in ((c["w"], w), (None, None)):
        c["Y"].fill_(float("nan"))
        L.logra_expert_combine(c["Ys"], c["slots"], c["Y"], weights=weights)
        ref, mag = ox.combine(_f64(c["Ys"]), slots, wr)
        assert np.all(np.abs(_f64(c["Y"]) - ref) <= half * np.abs(ref) + (1 + half) * (K + 1) * 2.0 ** -24 * mag + tiny)
    # gradient
    before = c["dYs"].clone()
    dw = torch.full((T, K), float("nan"), device=dev)
    L.logra_expert_combine_backward(c["dY"], c["Ys"], c["slots"], c["w"], c["dYs"], dw)
    ref, dwr, mag = ox.combine_backward(_f64(c["dY"]), _f64(c["Ys"]), slots, w, _f64(before))
    assert np.all(np.abs(_f64(c["dYs"]) - ref) <= (half + 2.0 ** -23) * np.abs(ref) + tiny)
    V = 8 if dt == torch.bfloat16 else 4
    chain = -(-h // (256 * V)) * V + 11
    assert np.all(np.abs(_f64(dw) - dwr) <= chain * 2.0 ** -24 * mag + tiny)
    kept = slots >= 0
    assert np.all(_f64(dw)[~kept] == 0)


@pytest.mark.parametrize("dt,raw", [(torch.bfloat16, torch.int16), (torch.float32, torch.int32)])
def test_gather_without_weights_copies_every_bit_pattern(dt, raw):
    dev = device()
    g = torch.Generator().manual_seed(0)
    lo, hi = torch.iinfo(raw).min, torch.iinfo(raw).max
    X = torch.randint(lo, hi, (33, 2003), generator=g, dtype=torch.int64).to(raw).to(dev)     # NaNs of every payload
    offsets, order, slots = _sort(_ids(5, 33, 3, 7).to(dev), 7, dev)
    Xs = torch.zeros(99, 2003, dtype=raw, device=dev)
    L.logra_expert_gather(X.view(dt), slots, Xs.view(dt))
    n = int(offsets[-1])
    assert torch.equal(Xs[:n], X[order[:n].long() // 3]) and not Xs[n:].any()


def test_gather_and_combine_are_each_others_gradient():
    """<combine(Ys, w), G> differentiated: by differences of the forward call
    (the function is linear in Ys and in w, so a difference over a step of 1/4
    is exact up to the rounding of its two values) and by the gradient call;
    the gather's gradient is combine."""
    dev = device()
    T, K, E, h = 12, 3, 5, 96
    c = _case(3, T, K, E, h, torch.float32, dev, drop=0.2)
    G = c["dY"].double()
    dYs, dw = torch.zeros_like(c["dYs"]), torch.zeros(T, K, device=dev)
    L.logra_expert_combine_backward(c["dY"], c["Ys"], c["slots"], c["w"], dYs, dw)

    def loss(Ys, w):
        Y = torch.empty(T, h, device=dev)
        L.logra_expert_combine(Ys, c["slots"], Y, weights=w)
        return float((Y.double() * G).sum())

    _, mag = ox.combine(_f64(c["Ys"]), c["slots"].cpu().numpy(), np.abs(_f64(c["w"])) + 0.25)
    tol = 2 * (K + 2) * 2.0 ** -24 * float((torch.from_numpy(mag).to(dev) * G.abs()).sum()) / 0.5
    for t, j in ((0, 0), (5, 2), (11, 1), (7, 0)):
        up, down = c["w"].clone(), c["w"].clone()
        up[t, j] += 0.25
        down[t, j] -= 0.25
        assert abs((loss(c["Ys"], up) - loss(c["Ys"], down)) / 0.5 - float(dw[t, j])) <= tol + 1e-5
    for s, col in ((0, 0), (3, 50), (20, 95)):
        up, down = c["Ys"].clone(), c["Ys"].clone()
        up[s, col] += 0.25
        down[s, col] -= 0.25
        assert abs((loss(up, c["w"]) - loss(down, c["w"])) / 0.5 - float(dYs[s, col])) <= tol + 1e-5
    # <gather(X), H> = <X, combine(H)>
    H = c["Ys"]
    Xs, dX = torch.zeros(T * K, h, device=dev), torch.empty(T, h, device=dev)
    L.logra_expert_gather(c["X"], c["slots"], Xs, weights=c["w"])
    L.logra_expert_combine(H, c["slots"], dX, weights=c["w"])
    a, b = float((Xs.double() * H.double()).sum()), float((c["X"].double() * dX.double()).sum())
    size = float((Xs.double().abs() * H.double().abs()).sum())
    assert abs(a - b) <= (K + 2) * 2.0 ** -24 * size * 2


def test_dropped_rows_and_non_finite_rows_stay_apart():
    dev = device()
    T, K, E, h = 20, 2, 4, 264
    for dt in (torch.bfloat16, torch.float32):
        c = _case(8, T, K, E, h, dt, dev, drop=0.4)
        kept = int(c["offsets"][-1])
        c["Ys"][kept:] = float("nan")                  # behind the last sorted row: never read
        c["dYs"][kept:] = 7.0
        Y, dw = torch.empty(T, h, dtype=dt, device=dev), torch.empty(T, K, device=dev)
        L.logra_expert_combine(c["Ys"], c["slots"], Y, weights=c["w"])
        assert torch.isfinite(Y).all()
        L.logra_expert_combine_backward(c["dY"], c["Ys"], c["slots"], c["w"], c["dYs"], dw)
        assert torch.isfinite(dw).all() and (c["dYs"][kept:] == 7.0).all()
        empty = (c["slots"] < 0).all(1)
        assert empty.any() and not Y[empty].any()
        # a slot outside the rows given counts as dropped
        L.logra_expert_combine(c["Ys"][:3], c["slots"], Y)
        ref, _ = ox.combine(_f64(c["Ys"]), np.where(c["slots"].cpu().numpy() < 3, c["slots"].cpu().numpy(), -1), None)
        assert np.all(np.abs(_f64(Y) - ref) <= 2.0 ** -7 * np.abs(ref) + 1e-30)
        # an infinite row reaches its own token only
        c["Ys"][0, 5] = float("inf")
        L.logra_expert_combine(c["Ys"], c["slots"], Y, weights=c["w"])
        t = int(c["order"][0]) // K
        assert not torch.isfinite(Y[t, 5]) and int((~torch.isfinite(Y)).sum()) == 1


def test_rows_past_32_bit_offsets():
    dev = device()
    T, K, E, h = 70000, 8, 32, 2048                    # 560000 rows of 4 KB: 2.3 GB
    ids = torch.randint(0, E, (T, K), generator=torch.Generator(device=dev).manual_seed(0), device=dev)
    offsets, order, slots = _sort(ids, E, dev)
    X = torch.randn(T, h, generator=torch.Generator(device=dev).manual_seed(1), device=dev).to(torch.bfloat16)
    Xs = torch.zeros(T * K, h, dtype=torch.bfloat16, device=dev)
    assert Xs.numel() * 2 > 1 << 31
    L.logra_expert_gather(X, slots, Xs)
    for a in range(0, T * K, 100000):
        assert torch.equal(Xs[a:a + 100000], X[order[a:a + 100000].long() // K])
    # eight equal copies of a bf16 row: every partial sum is the row times a small whole number
    Y, dw = torch.empty_like(X), torch.empty(T, K, device=dev)
    L.logra_expert_combine(Xs, slots, Y)
    assert torch.equal(Y.float(), 8 * X.float())
    w = torch.full((T, K), 0.5, device=dev)
    out = torch.zeros_like(Xs)
    L.logra_expert_combine_backward(X, Xs, slots, w, out, dw)
    for a in range(0, T * K, 100000):
        assert torch.equal(out[a:a + 100000].float(), 0.5 * Xs[a:a + 100000].float())
    sq = X.float().square().sum(1, keepdim=True)
    assert torch.all((dw - sq).abs() <= 64 * 2.0 ** -24 * sq)


def test_repeats_graph_and_side_stream():
    dev = device()
    T, K, E, h = 1100, 8, 40, 264                      # the sort in several workgroups
    c = _case(21, T, K, E, h, torch.bfloat16, dev)
    ids = _ids(21, T, K, E).to(dev)
    ws = torch.empty(max(1, L.logra_expert_sort_workspace_bytes(T, K, E)), dtype=torch.uint8, device=dev)
    off, order, slots = (torch.empty_like(c[n]) for n in ("offsets", "order", "slots"))
    Xs, dYs = torch.zeros(T * K, h, dtype=torch.bfloat16, device=dev), torch.zeros(T * K, h, dtype=torch.bfloat16, device=dev)
    Y, dw = torch.empty(T, h, dtype=torch.bfloat16, device=dev), torch.empty(T, K, device=dev)
    outs = (off, order, slots, Xs, Y, dYs, dw)

    def work(stream=None, ws=ws):
        L.logra_expert_sort(ids, E, off, order, slots, ws=ws, stream=stream)
        L.logra_expert_gather(c["X"], slots, Xs, stream=stream)
        L.logra_expert_combine(Xs, slots, Y, weights=c["w"], stream=stream)
        L.logra_expert_combine_backward(c["dY"], Xs, slots, c["w"], dYs, dw, stream=stream)

    work()
    torch.cuda.synchronize()
    _same_sort((off, order, slots), ids, E)
    ref = [o.clone() for o in outs]

    def same():
        torch.cuda.synchronize()
        for a, b in zip(outs, ref):
            assert torch.equal(a, b)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        for o in outs:
            o.zero_()
        side.wait_stream(torch.cuda.current_stream())
        work(stream=side, ws=None)
        same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(3):
        work()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        same()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("h", [9, 1499, 2047])
def test_infinities_near_a_row_end_off_the_vector_width(h, dt):
    """An infinity counts once wherever it stands: <dY, Ys> stays infinite, and
    no other element of the row is touched by it."""
    dev = device()
    T, K, E = 4, 3, 5
    offsets, order, slots = _sort(_ids(2, T, K, E).to(dev), E, dev)
    w = torch.full((T, K), 2.0, device=dev)
    for at in sorted({max(0, h - 1 - i) for i in range(10)}):
        dY = torch.ones(T, h, device=dev).to(dt)
        Ys = torch.ones(T * K, h, device=dev).to(dt)
        Ys[:, at] = float("inf")
        Y, dYs, dw = torch.empty_like(dY), torch.zeros_like(Ys), torch.empty(T, K, device=dev)
        L.logra_expert_combine(Ys, slots, Y, weights=w)
        L.logra_expert_combine_backward(dY, Ys, slots, w, dYs, dw)
        kept = slots >= 0
        assert torch.equal(dw.isinf(), kept) and not dw.isnan().any()
        some = kept.any(1)
        assert torch.equal(Y[some][:, at].float(), torch.full((int(some.sum()),), float("inf"), device=dev))
        rest = torch.arange(h, device=dev) != at
        assert torch.equal(Y[:, rest].float(), (2 * kept.sum(1, keepdim=True)).float().expand(T, h - 1))
