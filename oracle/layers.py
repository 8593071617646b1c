"""Plain numpy forms of routing, of 8-bit codes and their products, and of the
AdamW step with moments in 32 or 8 bits; for tests. Whatever the library must
reproduce bit by bit (codes, scales, ids) is formed here in the type that fixes
it, everything else in fp64."""
from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1
GOLDEN, MIX1, MIX2 = 0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB
ADAM_ID = 0xFFFFFFFFFFFFFFFF
BLOCK = 256


# ----------------------------------------------------------------- routing --
def scores(x, score):
    """Scores of rows of logits; -inf and NaN logits have none (0)."""
    x = np.asarray(x, np.float64)
    live = x > -np.inf
    with np.errstate(all="ignore"):
        if score == SIGMOID:
            return np.where(live, 1 / (1 + np.exp(-x)), 0.0)
        top = np.max(np.where(live, x, -np.inf), axis=1, keepdims=True)
        e = np.where(live, np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
        total = e.sum(1, keepdims=True)
        return e / np.where(total > 0, total, 1.0)


def route(x, topk, score, bias=None, groups=1, topk_groups=1, group_best=1, renormalize=True, scale=1.0):
    """(ids, weights) of rows of logits, choice by choice. A softmax with a logit
    of +inf has no values: choices are by the logits, weights NaN."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    s = scores(x, score)
    key = s + (0.0 if bias is None else np.asarray(bias, np.float64))
    if bias is None and not (groups > topk_groups and group_best == 2):
        key = x.copy()                          # sorts alike, also where scores are equal in 64 bits
    lost = (x == np.inf).any(1) & (score == SOFTMAX)
    if bias is not None:
        key[lost] = np.where(np.asarray(bias, np.float64) > -np.inf, x[lost], -np.inf)
    else:
        key[lost] = x[lost]
    key = np.where((x > -np.inf) & (key > -np.inf), key, -np.inf)
    ids, w = np.full((T, topk), -1), np.zeros((T, topk))
    for t in range(T):
        k = key[t].copy()
        if groups > topk_groups:
            parts = np.sort(k.reshape(groups, -1), axis=1)[:, ::-1][:, :group_best]
            rank = np.where(parts[:, 0] > -np.inf, np.where(parts > -np.inf, parts, 0.0).sum(1), -np.inf)
            kept = np.argsort(-rank, kind="stable")[:topk_groups]
            stays = np.isin(np.arange(E) // (E // groups), kept)
            k = np.where(stays, k, -np.inf)
        for j in range(topk):
            e = int(np.argmax(k))               # the first of equals
            if k[e] == -np.inf:
                break
            ids[t, j], w[t, j] = e, s[t, e]
            k[e] = -np.inf
        n = int((ids[t] >= 0).sum())
        if renormalize and n:
            if score == SIGMOID:                # ratios, also where every sigmoid vanishes in fp64
                c = x[t, ids[t, :n]]
                w[t, :n] = np.exp(np.minimum(c, 0) - min(c.max(), 0)) / (1 + np.exp(-np.abs(c)))
            w[t, :n] /= w[t, :n].sum()
        if np.isnan(x[t]).any() or lost[t]:
            w[t, :n] = np.nan
    return ids, scale * w


def route_weights(x, ids, score, renormalize, scale):
    """Weights of given ids (fp64), a differentiable function of the logits."""
    s = scores(x, score)
    ok = (ids >= 0) & (ids < s.shape[1])
    p = np.where(ok, np.take_along_axis(s, np.where(ok, ids, 0), 1), 0.0)
    if renormalize:
        total = p.sum(1, keepdims=True)
        p = p / np.where(total > 0, total, 1.0)
    return scale * p


def route_backward(x, ids, dw, score, renormalize, scale):
    """(dlogits, the sum of the magnitudes that its terms have)."""
    s = scores(x, score)
    T, E = s.shape
    ok = (ids >= 0) & (ids < E)
    at = np.where(ok, ids, 0)
    g = np.where(ok, scale * np.asarray(dw, np.float64), 0.0)
    p = np.where(ok, np.take_along_axis(s, at, 1), 0.0)
    if renormalize:
        total = p.sum(1, keepdims=True)
        total = np.where(total > 0, total, 1.0)
        dp = np.where(ok, g / total - (p * g).sum(1, keepdims=True) / total ** 2, 0.0)
        mp = np.where(ok, np.abs(g) / total + (p * np.abs(g)).sum(1, keepdims=True) / total ** 2, 0.0)
    else:
        dp, mp = g, np.abs(g)
    ds, ms = np.zeros((T, E)), np.zeros((T, E))
    for j in range(ids.shape[1]):
        np.add.at(ds, (np.arange(T), at[:, j]), dp[:, j])
        np.add.at(ms, (np.arange(T), at[:, j]), mp[:, j])
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            slope = s / (1 + np.exp(np.asarray(x, np.float64)))
        return ds * slope, ms * slope
    return (s * (ds - (s * ds).sum(1, keepdims=True)), s * (ms + (s * ms).sum(1, keepdims=True)))


# -------------------------------------------------------------------- e4m3 --
def e4m3_values():
    """The values of codes 0 .. 126 (127: NaN); code + 128: their negatives."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def decode(codes):
    v = np.append(e4m3_values(), np.nan)
    c = np.asarray(codes).astype(np.int64)
    return np.where(c >= 128, -1.0, 1.0) * v[c & 127]


def encode(q):
    """Codes of the values nearest to q (ties to the even code; at most 448)."""
    v = e4m3_values()
    q = np.asarray(q, np.float64)
    a = np.minimum(np.abs(q), 448.0)
    hi = np.searchsorted(v, a)                 # v[hi - 1] < a <= v[hi]
    hi = np.minimum(hi, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = v[hi] - a, a - v[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (v[hi] == a), hi, lo)
    code = np.where(np.isnan(q), 127, code)
    return (code | np.where(np.signbit(q), 128, 0)).astype(np.uint8)


def quantize(x, block_rows, transpose=False):
    """(codes, scales) of one array; quotients in fp32."""
    x = np.asarray(x, np.float32)
    n, k = x.shape
    rb, kb = -(-n // block_rows), -(-k // 128)
    scale = np.ones((rb, kb), np.float32)
    codes = np.zeros((n, k), np.uint8)
    with np.errstate(all="ignore"):
        for i in range(rb):
            for j in range(kb):
                part = x[i * block_rows:(i + 1) * block_rows, 128 * j:128 * (j + 1)]
                mags = np.abs(part)[~np.isnan(part)]
                s = np.float32(mags.max() if mags.size else 0) / np.float32(448)
                scale[i, j] = s if s > 0 else 1
                codes[i * block_rows:(i + 1) * block_rows, 128 * j:128 * (j + 1)] = encode(part / scale[i, j])
    return (codes.T.copy(), scale.T.copy()) if transpose else (codes, scale)


def dequantize(codes, scales, block_rows):
    n, k = codes.shape
    return decode(codes) * np.repeat(np.repeat(np.asarray(scales, np.float64), block_rows, 0)[:n], 128, 1)[:, :k]


def matmul(x, xs, w, ws, before, offsets=None, order=None, topk=1):
    """(Y, sums of magnitudes) of codes and scales; before: Y as it was."""
    xd = dequantize(x, xs, 1)
    if offsets is None:
        xd, wd = xd[:len(before)], dequantize(w, ws, 128)       # x may have more rows than Y
        return xd @ wd.T, np.abs(xd) @ np.abs(wd).T
    Y, mag = np.array(before, np.float64), np.zeros(before.shape)
    M = Y.shape[0]
    for e in range(w.shape[0]):
        a = min(max(int(offsets[e]), 0), M)
        b = min(max(int(offsets[e + 1]), a), M)
        rows = np.arange(a, b) if order is None else np.where(order[a:b] >= 0, order[a:b] // topk, -1)
        ok = (rows >= 0) & (rows < xd.shape[0])
        part = np.where(ok[:, None], xd[np.where(ok, rows, 0)], 0.0)
        wd = dequantize(w[e], ws[e], 128)
        Y[a:b], mag[a:b] = part @ wd.T, np.abs(part) @ np.abs(wd).T
    return Y, mag


def groups_largest(x, xs, w, ws, step=64):
    """Sum over the groups of eight neighbouring k of the largest product's
    magnitude (scaled): dense operands."""
    xd, wd = np.abs(dequantize(x, xs, 1)), np.abs(dequantize(w, ws, 128))
    pad = -xd.shape[1] % 8
    xd, wd = (np.pad(np.nan_to_num(t), ((0, 0), (0, pad))).reshape(len(t), -1, 8).astype(np.float32) for t in (xd, wd))
    out = np.zeros((len(xd), len(wd)))
    for a in range(0, len(xd), step):
        for g in range(xd.shape[1]):
            out[a:a + step] += (xd[a:a + step, None, g] * wd[None, :, g]).max(-1)
    return out


# ------------------------------------------------------------------- AdamW --
def _mix(z):
    z = (z ^ (z >> np.uint64(30))) * np.uint64(MIX1)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(MIX2)
    return z ^ (z >> np.uint64(31))


def chances(seed, step, n):
    """16-bit numbers of the n state elements: (for m, for the root)."""
    with np.errstate(over="ignore"):
        h = lambda x: _mix(np.uint64(x) + np.uint64(GOLDEN))  # noqa: E731
        key = h(h(h(np.array([seed], np.uint64)) ^ np.uint64(step)) ^ np.uint64(ADAM_ID))
        words = _mix(key + (np.arange(n // 2, dtype=np.uint64) + np.uint64(1)) * np.uint64(GOLDEN))
    parts = words.view(np.uint16).reshape(n, 2)
    return parts[:, 0].astype(np.int64), parts[:, 1].astype(np.int64)


def round_codes(x, u, floor=False):
    """(codes, scales) of fp32 values in blocks; u: their 16-bit numbers. floor:
    a value above zero keeps the smallest code."""
    x = np.asarray(x, np.float32).reshape(-1, BLOCK)
    u = u.reshape(-1, BLOCK)
    codes, scales = np.zeros(x.shape, np.uint8), np.zeros(len(x), np.float32)
    f = np.float32
    v = e4m3_values()
    for b in range(len(x)):
        if not np.isfinite(x[b]).all():
            scales[b] = np.nan
            continue
        top = np.abs(x[b]).max()
        live = top >= f(2.0) ** -100
        scales[b] = top / f(448) if live else 0
        a = np.minimum(np.abs(x[b]) * (f(448) / top if live else f(0)), f(448))
        # places of a among the codes' steps, and the chance added
        e = np.maximum(np.frexp(a)[1] - 1, -6)
        step = np.ldexp(f(1), e - 3).astype(f)
        q = np.floor(a / step + (u[b].astype(f) + f(0.5)) * f(2.0 ** -16)) * step
        c = np.searchsorted(v, q.astype(np.float64))
        if floor and live:
            c = np.where((x[b] > 0) & (c == 0), 1, c)
        codes[b] = c | np.where(np.signbit(x[b]), 128, 0)
    return codes.reshape(-1), scales


def adamw(p, g, m, v, lr, beta1, beta2, eps, wd, step, coef=1.0):
    """(p', m', v') in fp64, and (m', root) in fp32 in the library's order."""
    f = np.float32
    with np.errstate(all="ignore"):
        gc = np.asarray(g, f) * f(coef)
        m32 = f(beta1) * np.asarray(m, f) + f(1 - beta1) * gc
        v32 = f(beta2) * np.asarray(v, f) + f(1 - beta2) * (gc * gc)
        root = np.sqrt(v32)
        g64 = np.asarray(g, np.float64) * float(f(coef))
        m64 = beta1 * np.asarray(m, np.float64) + (1 - beta1) * g64
        v64 = beta2 * np.asarray(v, np.float64) + (1 - beta2) * g64 ** 2
        p64 = np.asarray(p, np.float64)
        upd = lr / (1 - beta1 ** step) * m64 / (np.sqrt(v64 / (1 - beta2 ** step)) + eps)
        return p64 - lr * wd * p64 - upd, m64, v64, m32, root
