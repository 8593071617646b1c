"""AdamW over lists of tensors against the plain form.

Tolerances. 8-bit codes, their scales and the 32-bit moments' fp32 sequence are
reproduced bit by bit. Against fp64: a moment is two products and a sum (three
roundings of terms of its own size: 2^-22 of their magnitudes); the parameter
takes the decay (two roundings), the update (moments, root, two quotients and
three products: 16 x 2^-24 of it, as m enters with its own 2^-22 of the terms'
magnitudes) and one rounding of the result (2^-24; bf16 2^-8)."""
import numpy as np
import pytest
import torch

import rank_gradient_sketching_sketch_amd as L
from oracle import layers as ox
from gpu_util import device, say

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
INF, NAN = float("inf"), float("nan")


def _np(t):
    return t.detach().float().cpu().numpy()


class Model:
    """Tensors of given shapes and types; rows of 2-D ones may have gaps, and every buffer an odd begin."""

    def __init__(self, seed, shapes, dev, p=F32, g=F32, c=None, gap=0, bits=32, state=True):
        gen = torch.Generator().manual_seed(seed)

        def tensor(shape, dt, std):
            if dt is None:
                return None
            if gap and len(shape) == 2:
                return (std * torch.randn(shape[0], shape[1] + gap, generator=gen)).to(dt).to(dev)[:, 1:1 + shape[1]]
            n = int(np.prod(shape))
            return (std * torch.randn(n + 1, generator=gen)).to(dt).to(dev)[1:].view(shape) if n else torch.zeros(shape, dtype=dt, device=dev)

        pick = lambda dt, i: dt[i % len(dt)] if isinstance(dt, tuple) else dt  # noqa: E731
        self.p = [tensor(s, pick(p, i), 0.5) for i, s in enumerate(shapes)]
        self.g = [tensor(s, pick(g, i), 0.1) for i, s in enumerate(shapes)]
        self.c = [tensor(s, pick(c, i), 1.0) for i, s in enumerate(shapes)]
        self.list = L.AdamWList(self.p, self.g, state_bits=bits, copies=self.c)
        if state:                       # moments as in the middle of a training
            used = torch.zeros(256 * self.list.blocks)
            for f, t in zip(self.list.first, self.p):
                used[256 * f:256 * f + t.numel()] = 1
            m = 0.05 * torch.randn(256 * self.list.blocks, generator=gen) * used
            r = 0.1 * torch.rand(256 * self.list.blocks, generator=gen) * used
            if bits == 32:
                self.list.exp_avg.copy_(m)
                self.list.exp_avg_sq.copy_(r * r)
            else:
                half = np.full(256 * self.list.blocks, 32768)
                for dst, x, row in ((self.list.exp_avg, m, 0), (self.list.exp_avg_sq, r, 1)):
                    codes, scales = ox.round_codes(x.numpy(), half)
                    dst.view(torch.uint8).copy_(torch.from_numpy(codes))
                    self.list.scales[row].copy_(torch.from_numpy(scales))

    def moments(self):
        """fp32 (m, v) that the state stands for."""
        l = self.list
        if l.state_bits == 32:
            return _np(l.exp_avg), _np(l.exp_avg_sq)
        m, r = ((_np(t).reshape(-1, 256) * _np(l.scales[i])[:, None]).reshape(-1) for i, t in enumerate((l.exp_avg, l.exp_avg_sq)))
        return m, r * r

    def flat(self, tensors):
        out = np.zeros(256 * self.list.blocks, np.float32)
        for f, t in zip(self.list.first, tensors):
            out[256 * f:256 * f + t.numel()] = _np(t).reshape(-1)
        return out


def _check_step(model, step, coef=1.0, seed=0, norm=None, max_norm=INF, hyper=HYPER):
    l = model.list
    m, v = model.moments()
    p, g = model.flat(model.p), model.flat(model.g)
    L.logra_adamw(l, hyper["lr"], hyper["beta1"], hyper["beta2"], hyper["eps"], hyper["weight_decay"], step, norm=norm,
                  max_norm=max_norm, seed=seed)
    p64, m64, v64, m32, root = ox.adamw(p, g, m, v, hyper["lr"], hyper["beta1"], hyper["beta2"], hyper["eps"], hyper["weight_decay"],
                                        step, coef)
    if l.state_bits == 32:
        assert np.array_equal(_np(l.exp_avg), m32)
        gm = np.abs(g.astype(np.float64) * coef)
        assert np.all(np.abs(_np(l.exp_avg) - m64) <= 2.0 ** -22 * (np.abs(m) + gm) + 1e-44)
        assert np.all(np.abs(_np(l.exp_avg_sq) - v64) <= 2.0 ** -22 * (np.abs(v) + gm ** 2) + 1e-44)
    else:
        um, ur = ox.chances(seed, step, 256 * l.blocks)
        for codes, scales, x, u, floor in ((l.exp_avg, l.scales[0], m32, um, False), (l.exp_avg_sq, l.scales[1], root, ur, True)):
            want, ws = ox.round_codes(x, u, floor)
            assert np.array_equal(scales.cpu().numpy(), ws, equal_nan=True)
            live = np.repeat(np.isfinite(ws), 256)
            assert np.array_equal(codes.view(torch.uint8).cpu().numpy()[live], want[live])
    with np.errstate(all="ignore"):
        terms = np.abs(m) + np.abs(g.astype(np.float64) * coef)
        slope = hyper["lr"] / (1 - hyper["beta1"] ** step) / (np.sqrt(v64 / (1 - hyper["beta2"] ** step)) + hyper["eps"])
    allowed = 16 * 2.0 ** -24 * slope * terms + 2.0 ** -22 * hyper["lr"] * abs(hyper["weight_decay"]) * np.abs(p) + 1e-44
    for f, t, c in zip(l.first, model.p, model.c):
        at = slice(256 * f, 256 * f + t.numel())
        for got in (t,) if c is None else (t, c):
            half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
            want = p64[at]
            assert np.all(np.abs(_np(got).reshape(-1) - want) <= half * np.abs(want) + (1 + half) * allowed[at])


SHAPES = [(3, 5), (256,), (257,), (0, 4), (1,), (64, 100), (1536,), (7, 1000), (0,), (2, 3, 37), (300, 1), (1, 900)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,g,c", [(F32, F32, None), (F32, BF, BF), (BF, BF, None), (BF, F32, F32), ((F32, BF), (BF, F32, F32), (None, BF, F32))])
@pytest.mark.parametrize("gap", [0, 3])
def test_steps(p, g, c, gap, bits):
    dev = device()
    say("adamw", p, g, c, gap, bits)
    model = Model(3, SHAPES, dev, p, g, c, gap, bits)
    for step in (7, 8):
        _check_step(model, step, seed=5)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_and_short_lists(bits):
    dev = device()
    for shapes in ([], [(0,)], [(1,)], [(5, 7), (0, 3)]):
        model = Model(1, shapes, dev, bits=bits, state=False)
        _check_step(model, 1)
    # the first step goes lr sign(g) far where the decay and eps are small
    p, g = torch.zeros(1000, device=dev), torch.randn(1000, generator=torch.Generator().manual_seed(1)).to(dev)
    L.logra_adamw(L.AdamWList([p], [g], state_bits=bits), 0.5, 0.9, 0.999, 1e-12, 0.0, 1)
    assert torch.allclose(p, -0.5 * g.sign(), rtol=1e-5, atol=0)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """Lists past one look of a wave (64, 4096 entries), and blocks past one launch's width."""
    dev = device()
    gen = np.random.default_rng(2)
    shapes = [(int(n),) for n in gen.integers(0, 700, 4200)]
    _check_step(Model(4, shapes, dev, g=BF, bits=bits), 3)
    _check_step(Model(5, [(40000, 257), (9,)], dev, bits=bits), 3)


@pytest.mark.parametrize("bits", [32, 8])
def test_norm(bits):
    dev = device()
    shapes = [(40, 30), (900,)]
    for norm, most, coef in ((4.0, 1.0, 0.25), (0.5, 1.0, 1.0), (3.0, INF, 1.0), (2.0, 0.0, 0.0), (7.0, 0.3, float(np.float32(0.3 / 7)))):
        _check_step(Model(6, shapes, dev, bits=bits), 4, coef=coef, norm=torch.tensor([norm], device=dev), max_norm=most)
    for bad in (INF, NAN):
        model = Model(6, shapes, dev, c=BF, bits=bits)
        l = model.list
        keep = [t.clone() for t in model.p + model.c + [l.exp_avg.view(torch.uint8), l.exp_avg_sq.view(torch.uint8)]]
        L.logra_adamw(l, 1e-3, 0.9, 0.99, 1e-8, 0.1, 4, norm=torch.tensor([bad], device=dev), max_norm=1.0)
        for a, b in zip(keep, model.p + model.c + [l.exp_avg.view(torch.uint8), l.exp_avg_sq.view(torch.uint8)]):
            assert torch.equal(a, b)
    # with the library's own norm, as a training step takes it
    model = Model(7, shapes, dev, bits=bits)
    norm = torch.empty(1, device=dev)
    L.logra_grad_norm(L.GradList(model.g), norm)
    _check_step(model, 2, coef=float(np.float32(0.5 / float(norm))), norm=norm, max_norm=0.5)


def test_values_that_are_not_finite_stay_in_their_block():
    dev = device()
    for bits in (32, 8):
        model = Model(8, [(1000,)], dev, bits=bits)
        clean = Model(8, [(1000,)], dev, bits=bits)
        model.g[0][300], model.g[0][301] = NAN, INF
        for m in (model, clean):
            L.logra_adamw(m.list, 1e-3, 0.9, 0.99, 1e-8, 0.0, 5)
        bad = ~torch.isfinite(model.p[0])
        assert bad.nonzero().reshape(-1).tolist() == [300, 301] and torch.equal(model.p[0][~bad], clean.p[0][~bad])
        a, b = model.moments()[0], clean.moments()[0]
        poisoned = ~np.isfinite(a)
        assert np.array_equal(np.flatnonzero(poisoned), [300, 301] if bits == 32 else np.arange(256, 512))
        assert np.array_equal(a[~poisoned], b[~poisoned])


def test_small_and_large_moments_in_8_bits():
    """Blocks that vanish, blocks near the largest and smallest magnitudes, one large value among small ones."""
    dev = device()
    model = Model(9, [(256 * 6,)], dev, bits=8, state=False)
    g = model.g[0]
    g[:256] = 0
    g[256:512] *= 1e-34
    g[512:768] *= 1e18
    g[768:1024] *= 1e-19
    g[1024] = 1e6
    for step in (1, 2, 3):
        _check_step(model, step)


@pytest.mark.parametrize("bits", [32, 8])
def test_resume_streams_and_graph(bits):
    dev = device()
    shapes = [(30, 70), (513,)]
    a, b = Model(10, shapes, dev, c=BF, bits=bits, state=False), Model(10, shapes, dev, c=BF, bits=bits, state=False)
    args = (1e-3, 0.9, 0.99, 1e-8, 0.1)
    for s in range(1, 5):
        L.logra_adamw(a.list, *args, s, seed=3)
    for s in (1, 2):
        L.logra_adamw(b.list, *args, s, seed=3)
    state = [t.clone() for t in (b.list.exp_avg, b.list.exp_avg_sq) + ((b.list.scales,) if bits == 8 else ())]
    again = L.AdamWList(b.p, b.g, state_bits=bits, copies=b.c, state=state)       # from a checkpoint
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (3, 4):
        L.logra_adamw(again, *args, s, seed=3, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(a.p + a.c + [a.list.exp_avg.view(torch.uint8)], b.p + b.c + [again.exp_avg.view(torch.uint8)]):
        assert torch.equal(x, y)
    assert again.describes(b.p, b.g, b.c) and not again.describes(b.p, b.g, None) and not again.describes(a.p, b.g, b.c)
    # a captured step, replayed on new gradients, against eager ones
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.logra_adamw(again, *args, 5, seed=3)
    for k in range(3):
        for t, u in zip(a.g, b.g):
            t.mul_(0.5).add_(0.01 * k)
            u.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        L.logra_adamw(a.list, *args, 5, seed=3)
        for x, y in zip(a.p + a.c + [a.list.exp_avg_sq.view(torch.uint8)], b.p + b.c + [again.exp_avg_sq.view(torch.uint8)]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_list_dropped_while_its_step_runs(bits):
    """The memory of table and state is not given to other tensors before the stream's step is over."""
    dev = device()
    model = Model(11, [(1 << 22,)], dev, bits=bits, state=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50000000)
    L.logra_adamw(model.list, 1e-3, 0.9, 0.99, 1e-8, 0.1, 1, stream=side)
    kept = [t for t in (model.list.table, model.list.exp_avg, model.list.exp_avg_sq, model.list.scales) if t is not None]
    old = {t.data_ptr() for t in kept}
    sizes = [t.numel() * t.element_size() for t in kept]
    model.list = None
    del kept
    new = [torch.full((n,), 255, dtype=torch.uint8, device=dev) for n in sizes]
    busy = not side.query()
    assert not busy or not old & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    assert busy and bool(torch.isfinite(model.p[0]).all())


def test_elements_past_32_bits():
    """A tensor of more than 2^31 elements, the second of its list: places at its ends and around 2^31 as in a list of their own."""
    dev = device()
    say("adamw past 32 bits")
    n, hyper = (1 << 31) + 3000, (1e-3, 0.9, 0.99, 1e-8, 0.1)
    g = torch.Generator(device=dev).manual_seed(3)
    p = torch.empty(n, device=dev).normal_(generator=g)
    d = torch.empty(n, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    spans = [(0, 1000), ((1 << 31) - 700, (1 << 31) + 800), (n - 1001, n)]
    small = [p[a:b].clone() for a, b in spans]
    grads = [d[a:b].clone() for a, b in spans]
    one, oned = torch.ones(5, device=dev), torch.ones(5, device=dev)
    big = L.AdamWList([one, p], [oned, d])
    few = L.AdamWList(small, grads)
    for step in (1, 2):
        L.logra_adamw(big, *hyper, step)
        L.logra_adamw(few, *hyper, step)
    for (a, b), t in zip(spans, small):
        assert torch.equal(p[a:b], t)
    assert not torch.equal(small[0], torch.ones_like(small[0])) and big.first == [0, 1]


def test_list_refusals():
    dev = device()
    p, g = torch.zeros(8, device=dev), torch.zeros(8, device=dev)
    for args, kw in ((([p], [p]), {}), (([p, p], [g, torch.zeros(8, device=dev)]), {}), (([p], [g[:7]]), {}), (([p], [g.half()]), {}),
                     (([p], [g.cpu()]), {}), (([p], [g]), dict(copies=[p])), (([p], [g]), dict(state=(p, g))),
                     (([p], [g]), dict(state_bits=8, state=(torch.zeros(256, device=dev), torch.zeros(256, device=dev)))),
                     (([torch.zeros(4, 4, device=dev).t()], [torch.zeros(4, 4, device=dev)]), {}),
                     (([torch.zeros(2, 3, 4, device=dev)[:, 1:]], [torch.zeros(2, 2, 4, device=dev)]), {})):
        with pytest.raises(L.LograError):
            L.AdamWList(*args, **kw)
    l = L.AdamWList([p], [g])
    for kw in (dict(step=0), dict(norm=torch.ones(2, device=dev)), dict(norm=torch.ones(1)), dict(max_norm=-1.0)):
        with pytest.raises(L.LograError):
            L.logra_adamw(l, 1e-3, 0.9, 0.99, 1e-8, 0.0, **{"step": 1, **kw})
