"""An expert layer's router and 8-bit products, the AdamW step of what is not sketched, and their measured cases.

Kinds (case["kind"]):
  route           top-k experts of every token from its logits (softmax or sigmoid scores, a bias for balance, groups of
                  experts, renormalised weights)
  route_backward  gradient of the weights carried back to the logits
  quantize        e4m3 codes with a scale for each 1 x 128 block of a row, or each 128 x 128 block of a weight
  matmul          Y = X W^T of such codes, dense or of the rows of every expert
  adamw           one AdamW step over many tensors with moments in 32 bits or in 8

Every kind works on seeded synthetic tensors. `own` selects between the plain torch form and the library.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 256                 # elements of an 8-bit moment's block
GOLDEN, MIX1, MIX2 = 0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB
ADAM_ID = 0xFFFFFFFFFFFFFFFF  # the matrix id whose counter stream the moments' rounding takes
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.01, 10


def listed():
    return [
        # the last token of a rollout: latency of the choice
        dict(name="route_1", kind="route", tokens=1, experts=128, topk=8, score="softmax", bias=False, groups=1, kept=1, best=1, renorm=True, dtype="f32", pad=0),
        # one microbatch of a 256-expert layer: sigmoid scores, a bias for balance, four of eight groups, padding tokens
        dict(name="route_4096", kind="route", tokens=4096, experts=256, topk=8, score="sigmoid", bias=True, groups=8, kept=4, best=2, renorm=True, dtype="f32", pad=130),
        # a ragged microbatch of a bf16 layer with few experts
        dict(name="route_backward_777", kind="route_backward", tokens=777, experts=60, topk=4, score="sigmoid", renorm=True, dtype="bf16", pad=20),
        # four microbatches at once, weights that are not renormalised: every logit has a gradient
        dict(name="route_backward_16384", kind="route_backward", tokens=16384, experts=128, topk=8, score="softmax", renorm=False, dtype="f32", pad=0),
        # activations of a ragged microbatch, a row that ends inside a block
        dict(name="quantize_rows_777", kind="quantize", batch=1, rows=777, cols=2064, block=1, turned=False, dtype="bf16"),
        # the weights of a 128-expert layer after an update, turned for the input gradient
        dict(name="quantize_experts", kind="quantize", batch=128, rows=768, cols=2048, block=128, turned=True, dtype="bf16"),
        # one token through the 7B up projection
        dict(name="matmul_1", kind="matmul", tokens=1, experts=0, topk=1, n=18944, k=3584, out="bf16", skew=0.0),
        # one microbatch through the 7B up projection
        dict(name="matmul_4096", kind="matmul", tokens=4096, experts=0, topk=1, n=18944, k=3584, out="bf16", skew=0.0),
        # one microbatch to 8 of 128 experts, read through the sorted order, uneven experts
        dict(name="matmul_experts", kind="matmul", tokens=4096, experts=128, topk=8, n=768, k=2048, out="bf16", skew=0.5),
        # the norm gains of the 28-layer 7B stack alone: launch-bound
        dict(name="adamw_gains", kind="adamw", rows=0, cols=3584, gains=57, bits=8, grad="bf16", copies=True, ratio=0.5),
        # an embedding and the gains of the 1.5B set, moments in 32 bits
        dict(name="adamw_32", kind="adamw", rows=32000, cols=1536, gains=57, bits=32, grad="f32", copies=False, ratio=0.0),
        # an embedding and the gains of the 7B set, moments in 8 bits, gradients clipped, the model's bf16 weights written too
        dict(name="adamw_8", kind="adamw", rows=32000, cols=3584, gains=57, bits=8, grad="bf16", copies=True, ratio=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("route", "route_backward", "quantize", "matmul", "adamw"))
    if kind in ("route", "route_backward"):
        groups = rng.choice((1, 1, 4, 8)) if kind == "route" else 1
        experts = groups * rng.randint(8, 256 // groups)
        tokens = _log(rng, 1, 16384)
        case = dict(kind=kind, tokens=tokens, experts=experts, topk=rng.choice((1, 2, 4, 6, 8)), score=rng.choice(("softmax", "sigmoid")),
                    renorm=rng.random() < 0.5, dtype=rng.choice(("f32", "bf16")), pad=rng.randint(0, tokens // 8))
        if kind == "route":
            case.update(bias=rng.random() < 0.5, groups=groups, kept=max(1, groups // 2), best=rng.choice((1, 2)))
        return case
    if kind == "quantize":
        block = rng.choice((1, 128))
        return dict(kind=kind, batch=rng.choice((1, 1, 8)), rows=_log(rng, 1, 2048), cols=16 * _log(rng, 4, 256), block=block,
                    turned=block == 128 and rng.random() < 0.5, dtype=rng.choice(("bf16", "f32")))
    if kind == "matmul":
        experts = rng.choice((0, 0, 8, 60))
        return dict(kind=kind, tokens=_log(rng, 1, 4096), experts=experts, topk=rng.choice((1, 2, 4)) if experts else 1,
                    n=_log(rng, 64, 2048 if experts else 8960), k=16 * _log(rng, 8, 128 if experts else 224),
                    out=rng.choice(("bf16", "bf16", "f32")), skew=rng.choice((0.0, 0.5, 1.0)) if experts else 0.0)
    copies = rng.random() < 0.5
    return dict(kind=kind, rows=_log(rng, 1, 16000), cols=rng.randint(64, 3600), gains=rng.randint(1, 60), bits=rng.choice((8, 32)),
                grad=rng.choice(("bf16", "f32")), copies=copies, ratio=rng.choice((0.0, 0.5, 3.0)))


# ------------------------------------------------------------------ inputs --
def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _logits(case, gen):
    x = 1.5 * torch.randn(case["tokens"], case["experts"], generator=gen, device=DEV) + 0.5 * torch.randn(case["experts"], generator=gen, device=DEV)
    if case["pad"]:
        x[case["tokens"] - case["pad"]:] = -math.inf        # padding tokens take no expert
    return x.to(_type(case["dtype"]))


def _codes(gen, *shape):
    """Codes as a quantiser leaves them, and scales of about one."""
    return (torch.randn(*shape, generator=gen, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)


def _scales(gen, std, *shape):
    return std / 100 * torch.exp2(torch.rand(*shape, generator=gen, device=DEV) - 0.5)


def _sizes(case):
    """Elements of every tensor of an AdamW step."""
    return [case["rows"] * case["cols"]] * (case["rows"] > 0) + [case["cols"]] * case["gains"]


def _starts(sizes):
    """Where every tensor begins in the flat buffers: at a block's begin."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    return at


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    kind, s = case["kind"], dict(case=case)
    if kind == "route":
        T, E = case["tokens"], case["experts"]
        s.update(logits=_logits(case, gen), ids=torch.empty(T, case["topk"], dtype=torch.int32, device=DEV),
                 weights=torch.empty(T, case["topk"], device=DEV),
                 bias=0.1 * torch.randn(E, generator=gen, device=DEV) if case["bias"] else None)
    elif kind == "route_backward":
        x = _logits(case, gen)
        top, ids = torch.topk(x.float(), case["topk"], dim=1)
        s.update(logits=x, ids=torch.where(top > -math.inf, ids, -1).int().contiguous(), dlogits=torch.empty_like(x),
                 dweights=torch.randn(ids.shape, generator=gen, device=DEV) * 1e-2)
    elif kind == "quantize":
        b, n, k, blk = case["batch"], case["rows"], case["cols"], case["block"]
        grid = (-(-k // 128), -(-n // blk)) if case["turned"] else (-(-n // blk), -(-k // 128))
        s.update(x=(0.02 * torch.randn(b, n, k, generator=gen, device=DEV) * torch.exp(torch.randn(b, n, 1, generator=gen, device=DEV))).to(_type(case["dtype"])),
                 codes=torch.empty(b, *((k, n) if case["turned"] else (n, k)), dtype=torch.float8_e4m3fn, device=DEV), scales=torch.empty(b, *grid, device=DEV))
    elif kind == "matmul":
        T, E, n, k = case["tokens"], case["experts"], case["n"], case["k"]
        kb, nb = -(-k // 128), -(-n // 128)
        s.update(x=_codes(gen, T, k), xs=_scales(gen, 1.0, T, kb), w=_codes(gen, max(1, E), n, k), ws=_scales(gen, 0.02, max(1, E), nb, kb))
        rows = T
        if E:
            topk = min(case["topk"], E)
            logits = torch.randn(T, E, generator=gen, device=DEV) + case["skew"] * torch.randn(E, generator=gen, device=DEV)
            flat = torch.topk(logits, topk, dim=1).indices.reshape(-1)
            key, order = torch.sort(flat, stable=True)
            rows = T * topk
            s.update(order=order.int(), topk=topk, offsets=torch.searchsorted(key, torch.arange(E + 1, device=DEV)).int())
            s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["y"] = torch.empty(rows, n, dtype=_type(case["out"]), device=DEV)
    else:
        sizes = _sizes(case)
        starts = _starts(sizes)
        total = starts[-1]
        used = torch.zeros(total + 1, device=DEV)
        used[starts[:-1]] += 1
        used[[a + b for a, b in zip(starts, sizes)]] -= 1
        used = torch.cumsum(used[:-1], 0)               # one in a tensor, zero between two

        def made(std):
            return torch.randn(total, generator=gen, device=DEV).mul_(std).mul_(used)

        s.update(p=made(0.02), g=made(1e-2).to(_type(case["grad"])), copy=torch.zeros(total, dtype=torch.bfloat16, device=DEV) if case["copies"] else None)
        m, v = made(2e-3), made(1e-2).square_()
        if case["bits"] == 8:
            s["scales"] = torch.empty(2, total // BLOCK, device=DEV)
            s["m"], s["scales"][0] = _encode(m, 0.5)
            s["v"], s["scales"][1] = _encode(torch.sqrt(v), 0.5)
        else:
            s["m"], s["v"] = m, v
        norm = 1e-2 * math.sqrt(sum(sizes))
        s["norm"] = torch.full((1,), norm, device=DEV) if case["ratio"] else None
        s["max_norm"] = norm / case["ratio"] if case["ratio"] else math.inf
        s["sizes"], s["starts"] = sizes, starts
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program makes once for its tensors."""
    import rank_gradient_sketching_sketch_amd as L

    case = s["case"]
    if case["kind"] == "adamw":
        shapes = [(case["rows"], case["cols"])] * (case["rows"] > 0) + [(case["cols"],)] * case["gains"]

        def views(flat):
            return [flat[a:a + n].view(shape) for a, n, shape in zip(s["starts"], s["sizes"], shapes)]

        state = (s["m"], s["v"]) + ((s["scales"],) if case["bits"] == 8 else ())
        s["list"] = L.AdamWList(views(s["p"]), views(s["g"]), state_bits=case["bits"], copies=views(s["copy"]) if case["copies"] else None, state=state)


# --------------------------------------------------------------------- run --
def run(s):
    if own:
        return _run_own(s)
    return {"route": _route, "route_backward": _route_backward, "quantize": _quantize, "matmul": _matmul, "adamw": _adamw}[s["case"]["kind"]](s)


def _run_own(s):
    import rank_gradient_sketching_sketch_amd as L
    from rank_gradient_sketching_sketch_amd import binding as B

    case, kind = s["case"], s["case"]["kind"]
    if kind == "route":
        L.logra_route(s["logits"], s["ids"], s["weights"], bias=s["bias"], score=B.LOGRA_SIGMOID if case["score"] == "sigmoid" else B.LOGRA_SOFTMAX,
                      groups=case["groups"], topk_groups=case["kept"], group_best=case["best"], renormalize=case["renorm"], scale=2.5)
        return {"ids": s["ids"], "weights": s["weights"]}
    if kind == "route_backward":
        L.logra_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=B.LOGRA_SIGMOID if case["score"] == "sigmoid" else B.LOGRA_SOFTMAX,
                               renormalize=case["renorm"], scale=2.5)
        return {"dlogits": s["dlogits"]}
    if kind == "quantize":
        L.logra_fp8_quantize(s["x"], s["codes"], s["scales"], block_rows=case["block"], transpose=case["turned"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if kind == "matmul":
        if case["experts"]:
            L.logra_fp8_matmul(s["x"], s["xs"], s["w"], s["ws"], s["y"], offsets=s["offsets"], order=s["order"], topk=s["topk"])
        else:
            L.logra_fp8_matmul(s["x"], s["xs"], s["w"][0], s["ws"][0], s["y"])
        return {"y": s["y"]}
    L.logra_adamw(s["list"], LR, BETA1, BETA2, EPS, DECAY, STEP, norm=s["norm"], max_norm=s["max_norm"])
    return _state(s)


def _state(s):
    got = {"p": s["p"], "m": s["m"], "v": s["v"]}
    if s["case"]["bits"] == 8:
        got["scales"] = s["scales"]
    if s["copy"] is not None:
        got["copy"] = s["copy"]
    return got


def _route(s):
    case, x = s["case"], s["logits"].double()
    live = x > -math.inf
    score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1).nan_to_num(0.0)
    summed = case["groups"] > 1 and case["best"] > 1
    # without a bias and sums of keys a score and its logit sort alike
    key = score + s["bias"].double() if s["bias"] is not None else score if summed else x
    key = torch.where(live, key, -math.inf)
    if case["groups"] > 1:
        parts = key.view(x.shape[0], case["groups"], -1)
        best = torch.sort(parts, dim=2, descending=True).values[..., :case["best"]]
        found = best[..., 0] > -math.inf
        group = torch.where(found, torch.where(best > -math.inf, best, 0.0).sum(-1), -math.inf)
        kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        mask = torch.zeros_like(group, dtype=torch.bool).scatter_(1, kept, True)
        key = torch.where(mask[..., None], parts, -math.inf).view_as(key)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    top, ids = top[:, :case["topk"]], ids[:, :case["topk"]]
    chosen = top > -math.inf
    w = torch.where(chosen, score.gather(1, ids), 0.0)
    if case["renorm"]:
        w = w / torch.where(chosen.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
    return {"ids": torch.where(chosen, ids, -1).int(), "weights": (2.5 * w).float()}


def _route_backward(s):
    case, x = s["case"], s["logits"].float()
    chosen = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    dw = torch.where(chosen, 2.5 * s["dweights"], 0.0)
    if case["score"] == "sigmoid":
        p = torch.where(chosen, torch.sigmoid(x.gather(1, ids)), 0.0)
        slope = torch.where(chosen, torch.sigmoid(-x.gather(1, ids)), 0.0) * p
    else:
        score = torch.softmax(x, 1).nan_to_num(0.0)
        p = torch.where(chosen, score.gather(1, ids), 0.0)
        slope = p
    if case["renorm"]:
        total = torch.where(chosen.any(1, keepdim=True), p.sum(1, keepdim=True), 1.0)
        q = slope / total * (dw - (p / total * dw).sum(1, keepdim=True))
    else:
        q = slope * dw
    # choices that are none write to a column behind the last
    dx = torch.zeros(x.shape[0], x.shape[1] + 1, device=x.device).scatter_(1, torch.where(chosen, ids, x.shape[1]), q)[:, :-1]
    if case["score"] == "softmax" and not case["renorm"]:
        dx = dx - score * q.sum(1, keepdim=True)
    return {"dlogits": dx.to(s["logits"].dtype)}


def _blocks(x, size, dim):
    """Dimension dim in blocks of `size`, zeros behind the end."""
    n = x.shape[dim]
    pad = [0, 0] * (x.dim() - 1 - dim % x.dim()) + [0, -n % size]
    return torch.nn.functional.pad(x, pad).unflatten(dim, (-1, size))


def _quantize(s):
    case, x = s["case"], s["x"].float()
    b, n, k = x.shape
    blocks = _blocks(_blocks(x, 128, 2), case["block"], 1)        # b, n / block, block, k / 128, 128
    amax = blocks.abs().amax(dim=(2, 4), keepdim=True)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), 1.0)
    q = (blocks / scale).clamp(-448, 448).flatten(3, 4).flatten(1, 2)[:, :n, :k]
    scale = scale[:, :, 0, :, 0]
    if case["turned"]:
        q, scale = q.transpose(1, 2), scale.transpose(1, 2)
    return {"codes": q.to(torch.float8_e4m3fn).contiguous(), "scales": scale.contiguous()}


def _dense(s):
    """Activations and weights in 32 bits."""
    k, n = s["case"]["k"], s["case"]["n"]
    x = (_blocks(s["x"].float(), 128, 1) * s["xs"][..., None]).flatten(1)[:, :k]
    w = _blocks(_blocks(s["w"].float(), 128, 2), 128, 1) * s["ws"][:, :, None, :, None]
    return x, w.flatten(3, 4).flatten(1, 2)[:, :n, :k]


def _matmul(s):
    x, w = _dense(s)
    if not s["case"]["experts"]:
        return {"y": (x @ w[0].t()).to(s["y"].dtype)}
    counts = (s["offsets"][1:] - s["offsets"][:-1]).long()
    place = torch.arange(s["most"], device=x.device)
    slot = (s["offsets"][:-1, None] + place).long()                     # E x (rows of the longest expert)
    live = place[None, :] < counts[:, None]
    rows = s["order"].long()[torch.where(live, slot, 0)] // s["topk"]
    y = torch.bmm(x[rows], w.transpose(1, 2).contiguous())
    return {"y": y[live].to(s["y"].dtype)}                              # expert by expert: the sorted rows


def _i64(x):
    return x - (1 << 64) if x >= (1 << 63) else x


def _shr(z, n):
    return (z >> n) & ((1 << (64 - n)) - 1)


def _finalize(z):
    z = (z ^ _shr(z, 30)) * _i64(MIX1)
    z = (z ^ _shr(z, 27)) * _i64(MIX2)
    return z ^ _shr(z, 31)


def _uniforms(n, device):
    """16-bit uniform numbers of the step's counter stream, two an element (for m and for sqrt v): 2 x n, in [0, 1)."""
    g = _i64(GOLDEN)
    key = _finalize((_finalize(torch.zeros(1, dtype=torch.int64, device=device) + g) ^ STEP) + g)
    key = _finalize((key ^ _i64(ADAM_ID)) + g)
    words = _finalize(key + (torch.arange(n // 2, device=device) + 1) * g)      # one for two elements
    parts = (words[:, None] >> torch.arange(0, 64, 16, device=device)) & 0xFFFF
    return ((parts.view(-1, 2).float() + 0.5) / 65536).t()


def _pow2(e):
    return ((e + 127) << 23).int().view(torch.float32)


def _encode(x, u):
    """x in blocks of 256 as e4m3 codes and a scale, a block's largest at 448 of it, each value rounded up or down at the
    chance u of its place between two codes (u = 1/2: to nearest)."""
    x = x.view(-1, BLOCK)
    amax = x.abs().amax(1, keepdim=True)
    live = amax >= 2.0 ** -100
    most = torch.full_like(amax, 448.0)
    scale = torch.where(live, amax / most, 0.0)
    a = (x.abs() * torch.where(live, most / amax, 0.0)).clamp(max=448)
    e = torch.frexp(a)[1].clamp(min=-5) - 4                             # 2^-3 of a's binade, 2^-9 at least
    q = torch.floor(a * _pow2(-e) + (u.reshape(-1, BLOCK) if torch.is_tensor(u) else u)) * _pow2(e)
    return torch.copysign(q, x).to(torch.float8_e4m3fn).view(-1), scale[:, 0]


def _adamw(s):
    case = s["case"]
    g = s["g"].float()
    if s["norm"] is not None:
        g = g * torch.where(s["norm"] > s["max_norm"], s["max_norm"] / s["norm"].double(), 1.0).float()
    if case["bits"] == 8:
        m, r = ((s[a].float().view(-1, BLOCK) * s["scales"][i][:, None]).view(-1) for i, a in enumerate(("m", "v")))
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    root = torch.sqrt(v)
    upd = LR / (1 - BETA1 ** STEP) * (m / (root / math.sqrt(1 - BETA2 ** STEP) + EPS))
    s["p"].sub_(LR * DECAY * s["p"] + upd)
    if s["copy"] is not None:
        s["copy"].copy_(s["p"])
    if case["bits"] == 8:
        u = _uniforms(m.numel(), m.device)
        codes, s["scales"][0] = _encode(m, u[0])
        s["m"].copy_(codes)
        codes, s["scales"][1] = _encode(root, u[1])
        # the smallest code above zero for a root that is not zero
        s["v"].copy_(torch.where((root > 0) & (codes.float() == 0) & (s["scales"][1] > 0).repeat_interleave(BLOCK), 2.0 ** -9, codes.float()).to(codes.dtype))
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _state(s)


# -------------------------------------------------------------------- work --
def work(case):
    kind, el = case["kind"], {"bf16": 2, "f32": 4}
    if kind in ("route", "route_backward"):
        T, E, K, b = case["tokens"], case["experts"], case["topk"], el[case["dtype"]]
        live = T - case["pad"]
        if kind == "route":
            return {"bytes": b * T * E + 8 * T * K + 4 * E * case["bias"], "flops": 5 * live * E}
        whole = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": b * T * E + b * (live * E if whole else live * K) + 8 * T * K, "flops": 5 * live * (E if whole else K)}
    if kind == "quantize":
        b, n, k = case["batch"], case["rows"], case["cols"]
        return {"bytes": b * (n * k * (el[case["dtype"]] + 1) + 4 * -(-n // case["block"]) * -(-k // 128)), "flops": 3 * b * n * k}
    if kind == "matmul":
        T, n, k = case["tokens"], case["n"], case["k"]
        rows = T * (min(case["topk"], case["experts"]) if case["experts"] else 1)
        used = min(max(1, case["experts"]), rows)
        kb, nb = -(-k // 128), -(-n // 128)
        return {"bytes": T * (k + 4 * kb) + used * (n * k + 4 * nb * kb) + el[case["out"]] * rows * n + (4 * rows if case["experts"] else 0), "flops": 2 * rows * n * k}
    n = sum(_sizes(case))
    each = 8 + el[case["grad"]] + (4 if case["bits"] == 8 else 16) + 2 * case["copies"]
    return {"bytes": n * each + (16 * _starts(_sizes(case))[-1] // BLOCK if case["bits"] == 8 else 0), "flops": 14 * n}


# ------------------------------------------------------------------- exact --
def _e4m3(a):
    """Nearest e4m3 value of a >= 0 (at most 448), ties to even, in 64 bits."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(a.clamp(min=2.0 ** -30))), min=-6) - 3)
    return torch.round(a / step) * step


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"route": _exact_route, "route_backward": _exact_route_backward, "quantize": _exact_quantize, "matmul": _exact_matmul, "adamw": _exact_adamw}[case["kind"]](case, s)


def _exact_route(case, s):
    x = s["logits"].double()
    live = torch.isfinite(x)
    if case["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    key = score + (0 if s["bias"] is None else s["bias"].double())
    key = torch.where(live, key, -math.inf)
    T, E = x.shape
    G = case["groups"]
    out = torch.arange(E, device=DEV) // (E // G)
    if G > 1:
        total = torch.full((T, G), -math.inf, dtype=torch.float64, device=DEV)
        for g in range(G):          # group by group
            left = key[:, out == g].clone()
            for j in range(case["best"]):
                top, at = left.max(1)
                total[:, g] = torch.where(torch.isfinite(top), torch.where(torch.isfinite(total[:, g]), total[:, g], 0.0) + top, total[:, g])
                left.scatter_(1, at[:, None], -math.inf)
        allowed = torch.zeros(T, G, dtype=torch.bool, device=DEV)
        for _ in range(case["kept"]):
            best = total.amax(1, keepdim=True)
            at = (total == best).int().argmax(1, keepdim=True)
            allowed.scatter_(1, at, True)
            total.scatter_(1, at, -math.inf)
        key = torch.where(allowed[:, out], key, -math.inf)
    ids, w = [], []
    for _ in range(case["topk"]):   # choice by choice
        best = key.amax(1, keepdim=True)
        at = (key == best).int().argmax(1, keepdim=True)
        none = ~torch.isfinite(best)
        ids.append(torch.where(none, -1, at))
        w.append(torch.where(none, 0.0, score.gather(1, at)))
        key.scatter_(1, at, -math.inf)
    w = torch.cat(w, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return {"ids": torch.cat(ids, 1).int(), "weights": 2.5 * w}


def _exact_route_backward(case, s):
    """By the chain rule, choice by choice."""
    x = s["logits"].double()
    if case["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    at, chosen = s["ids"].long().clamp(min=0), s["ids"] >= 0
    dw = 2.5 * s["dweights"].double() * chosen
    p = score.gather(1, at) * chosen
    if case["renorm"]:
        total = p.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        dp = dw / total - (p * dw).sum(1, keepdim=True) / total.square()
    else:
        dp = dw
    dscore = torch.zeros_like(x)
    for j in range(at.shape[1]):
        dscore.scatter_add_(1, at[:, j:j + 1], (dp * chosen)[:, j:j + 1])
    if case["score"] == "sigmoid":
        return {"dlogits": dscore * score / (1 + torch.exp(x))}
    return {"dlogits": score * (dscore - (score * dscore).sum(1, keepdim=True))}


def _exact_quantize(case, s):
    b, n, k = s["x"].shape
    x = s["x"].double()
    codes, scales = torch.empty_like(x), []
    for j in range(0, k, 128):      # column block by column block
        part = x[:, :, j:j + 128]
        top = part.abs().amax(2)
        if case["block"] > 1:
            top = torch.stack([top[:, i:i + case["block"]].amax(1) for i in range(0, n, case["block"])], 1)
        scale = torch.where(top > 0, top / 448, 1.0)
        scales.append(scale)
        each = scale.repeat_interleave(case["block"], 1)[:, :n, None]
        codes[:, :, j:j + 128] = torch.sign(part) * _e4m3(part.abs() / each)
    scales = torch.stack(scales, 2)
    if case["turned"]:
        codes, scales = codes.transpose(1, 2), scales.transpose(1, 2)
    return {"codes": codes.contiguous(), "scales": scales.contiguous()}


def _exact_matmul(case, s):
    k, n, E = case["k"], case["n"], case["experts"]
    col = torch.arange(k, device=DEV) // 128
    row = torch.arange(n, device=DEV) // 128
    x = s["x"].double() * s["xs"].double()[:, col]
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    for e in range(max(1, E)):
        w = s["w"][e].double() * s["ws"][e].double()[row][:, col]
        if not E:
            y = x @ w.t()
        else:
            a, b = int(s["offsets"][e]), int(s["offsets"][e + 1])
            y[a:b] = x[s["order"][a:b].long() // s["topk"]] @ w.t()
    return {"y": y}


def _exact_code(x, u):
    """e4m3 codes and scales of x in blocks, in 64 bits, by logarithms."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    live = top >= 2.0 ** -100
    scale = torch.where(live, top / 448, 0.0)
    a = torch.where(live, x.abs() / torch.where(live, scale, 1.0), 0.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return (torch.sign(x) * torch.floor(a / step + u.double().reshape(-1, BLOCK)) * step).clamp(-448, 448).view(-1), scale[:, 0]


def _exact_adamw(case, s):
    g = s["g"].double()
    if s["norm"] is not None:
        norm = float(s["norm"])
        g = g * (s["max_norm"] / norm if norm > s["max_norm"] else 1.0)
    if case["bits"] == 8:
        each = s["scales"].double().repeat_interleave(BLOCK, 1)
        m, v = s["m"].double() * each[0], (s["v"].double() * each[1]).square()
    else:
        m, v = s["m"].double(), s["v"].double()
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g.square() * (1 - BETA2)
    mhat, vhat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
    p = s["p"].double() * (1 - LR * DECAY) - LR * mhat / (vhat.sqrt() + EPS)
    got = {"p": p, "m": m, "v": v}
    if case["bits"] == 8:
        u = _uniforms(m.numel(), m.device)
        got["m"], one = _exact_code(m, u[0])
        got["v"], two = _exact_code(v.sqrt(), u[1])
        got["v"] = torch.where((got["v"] == 0) & (v > 0) & (two > 0).repeat_interleave(BLOCK), 2.0 ** -9, got["v"])
        got["scales"] = torch.stack([one, two])
    if s["copy"] is not None:
        got["copy"] = p
    return got
