"""The operators around the sketch of an expert layer, and their measured cases.

Kinds (case["kind"]):
  clip              global L2 norm over many gradients (sketches in fp32, dense gradients in bf16) and the
                    clipped gradients
  dispatch          (token, choice) pairs sorted by expert, and the tokens' rows copied to their sorted places
  combine           the experts' rows weighted and summed back per token
  combine_backward  gradient of combine: the experts' rows' gradients and the weights' gradients
  sketch            S_e = dY_e^T (X_e A_e^T) for every expert e, X read through the sorted order

Every kind works on seeded synthetic tensors. `own` selects between the plain torch form and the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GOLDEN = 0x9E3779B97F4A7C15
MIX1, MIX2 = 0xBF58476D1CE4E5B9, 0x94D049BB133111EB
SEED, STEP, FIRST_ID = 0, 3, 70       # the sign matrices' key: library seed, optimizer step, expert 0's matrix id

# (d, k) of the seven projections of a layer, in the repository's workloads
LAYER_1_5B = ((1536, 1536), (256, 1536), (256, 1536), (1536, 1536), (8960, 1536), (8960, 1536), (1536, 8960))
LAYER_7B = ((3584, 3584), (512, 3584), (512, 3584), (3584, 3584), (18944, 3584), (18944, 3584), (3584, 18944))
SETS = {"1.5b": LAYER_1_5B, "7b": LAYER_7B}


def listed():
    return [
        # the unsketched gradients of a few layers alone (norm gains): a handful of short tensors, launch-bound
        dict(name="clip_gains", kind="clip", set="1.5b", layers=0, gains=9, r=256, odd=0, ratio=2.0),
        # one layer's seven sketches and its gains, gradients too large by a factor of four
        dict(name="clip_1.5b_layer", kind="clip", set="1.5b", layers=1, gains=2, r=256, odd=3, ratio=4.0),
        # the whole 28-layer 7B stack: 196 sketches, 1.42 GB, clipped
        dict(name="clip_7b_28layer", kind="clip", set="7b", layers=28, gains=57, r=256, odd=0, ratio=1.3),
        # a rollout's last few tokens: latency of the sort and the copy
        dict(name="dispatch_16", kind="dispatch", tokens=16, topk=8, experts=128, hidden=2048, dtype="bf16", pad=0, skew=1.0),
        # one microbatch with padding tokens at its end
        dict(name="dispatch_4096", kind="dispatch", tokens=4096, topk=8, experts=128, hidden=2048, dtype="bf16", pad=130, skew=0.5),
        # one token alone
        dict(name="combine_1", kind="combine", tokens=1, topk=8, experts=128, hidden=2048, dtype="bf16", pad=0, skew=0.5),
        # one microbatch, the ordinary training shape
        dict(name="combine_4096", kind="combine", tokens=4096, topk=8, experts=128, hidden=2048, dtype="bf16", pad=0, skew=0.5),
        # fp32 layer, two experts a token, ragged token count and a row length off every vector width
        dict(name="combine_backward_777", kind="combine_backward", tokens=777, topk=2, experts=8, hidden=1499, dtype="f32", pad=20, skew=1.0),
        # one microbatch, the ordinary training shape
        dict(name="combine_backward_4096", kind="combine_backward", tokens=4096, topk=8, experts=128, hidden=2048, dtype="bf16", pad=130, skew=0.5),
        # a small layer at the repository's small projection, few tokens per expert and empty experts
        dict(name="sketch_64", kind="sketch", tokens=64, topk=2, experts=16, d=256, k=1536, r=64, dtype="bf16", pad=3, skew=1.0),
        # the fp32 path at the repository's fp32 projection
        dict(name="sketch_f32", kind="sketch", tokens=384, topk=2, experts=8, d=256, k=512, r=32, dtype="f32", pad=0, skew=0.5),
        # one microbatch of a 128-expert layer (up projection of 768 features), uneven experts
        dict(name="sketch_4096", kind="sketch", tokens=4096, topk=8, experts=128, d=768, k=2048, r=256, dtype="bf16", pad=130, skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("clip", "dispatch", "combine", "combine_backward", "sketch"))
    if kind == "clip":
        which = rng.choice(("1.5b", "7b"))
        return dict(kind=kind, set=which, layers=rng.randint(0, 4 if which == "1.5b" else 12), gains=rng.randint(1, 60),
                    r=rng.choice((32, 64, 128, 256)), odd=rng.randint(0, 7), ratio=rng.choice((0.5, 1.5, 10.0)))
    experts = rng.choice((8, 16, 60, 64, 128, 256))
    topk = rng.choice((1, 2, 4, 6, 8))
    tokens = _log(rng, 1, 4096)
    case = dict(kind=kind, tokens=tokens, topk=topk, experts=experts, dtype=rng.choice(("bf16", "bf16", "f32")),
                pad=rng.randint(0, tokens // 8), skew=rng.choice((0.0, 0.5, 1.0, 2.0)))
    if kind == "sketch":
        if case["dtype"] == "f32":
            return dict(case, tokens=_log(rng, 1, 500), pad=0, experts=rng.choice((4, 8)), topk=rng.choice((1, 2)),
                        d=rng.randint(40, 256), k=rng.randint(40, 512), r=rng.choice((16, 32, 40)))
        return dict(case, experts=min(experts, 128), d=8 * _log(rng, 16, 96), k=8 * _log(rng, 32, 256),
                    r=rng.choice((32, 64, 128, 256)))
    hidden = rng.choice((_log(rng, 64, 2048), 8 * _log(rng, 16, 256)))
    return dict(case, hidden=min(hidden, 2048 if case["dtype"] == "bf16" else 1024))


# ------------------------------------------------------------------ inputs --
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _clip_shapes(case):
    sketches = [(d, case["r"]) for _ in range(case["layers"]) for d, _ in SETS[case["set"]]]
    gain = SETS[case["set"]][0][1] + case["odd"]
    return sketches, [(gain,)] * case["gains"]


def _routing(case, gen):
    """Expert ids (T x K, distinct per token, popular experts taken more often; -1 for padding tokens) and weights."""
    T, K, E = case["tokens"], min(case["topk"], case["experts"]), case["experts"]
    logits = torch.randn(T, E, generator=gen, device=DEV) + case["skew"] * torch.randn(E, generator=gen, device=DEV)
    top, ids = torch.topk(logits, K, dim=1)
    weights = torch.softmax(top, dim=1).contiguous()
    if case["pad"]:
        ids[T - case["pad"]:] = -1
    return ids.to(torch.int32).contiguous(), weights


def _slots_of(ids, experts):
    """Sorted place of every pair, on the host: what a program holds after the dispatch."""
    key = ids.reshape(-1).cpu().numpy().astype(np.int64)
    key = np.where((key < 0) | (key >= experts), experts, key)
    order = np.argsort(key, kind="stable")
    slots = np.empty(key.size, np.int32)
    slots[order] = np.arange(key.size, dtype=np.int32)
    slots[key == experts] = -1
    bounds = np.searchsorted(key[order], np.arange(experts + 1)).astype(np.int32)
    order = np.where(np.arange(key.size) < bounds[-1], order, -1).astype(np.int32)
    return (torch.from_numpy(slots).reshape(ids.shape).to(DEV), torch.from_numpy(order).to(DEV),
            torch.from_numpy(bounds).to(DEV), bounds)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    state = dict(case=case)
    if case["kind"] == "clip":
        sketches, gains = _clip_shapes(case)
        n_s, n_g = sum(a * b for a, b in sketches), sum(a for a, in gains)
        # one buffer per type, as a training program keeps its gradients; the tensors are views of it
        state["flat"] = {"sketch": torch.randn(n_s, generator=gen, device=DEV) * 1e-3,
                         "dense": (torch.randn(n_g, generator=gen, device=DEV) * 1e-2).to(torch.bfloat16)}
        state["out"] = {k: torch.zeros_like(v) for k, v in state["flat"].items()}
        expected = math.sqrt(n_s * 1e-6 + n_g * 1e-4)
        state["max_norm"] = float(np.float32(expected / case["ratio"]))
        state["norm"] = torch.zeros(1, device=DEV)
        state["coef"] = torch.zeros(1, device=DEV)
        if own:
            import rank_gradient_sketching_sketch_amd as L

            def views(flat):
                got, at = [], 0
                for s in sketches:
                    got.append(flat["sketch"][at:at + s[0] * s[1]].view(s))
                    at += s[0] * s[1]
                at = 0
                for s in gains:
                    got.append(flat["dense"][at:at + s[0]])
                    at += s[0]
                return got

            state["list"], state["out_list"] = L.GradList(views(state["flat"])), L.GradList(views(state["out"]))
        return state
    dt = _dtype(case)
    ids, weights = _routing(case, gen)
    T, K = ids.shape
    slots, order, offsets, bounds = _slots_of(ids, case["experts"])
    if case["kind"] == "dispatch":
        state.update(ids=ids, X=torch.randn(T, case["hidden"], generator=gen, device=DEV).to(dt),
                     Xs=torch.zeros(T * K, case["hidden"], dtype=dt, device=DEV),
                     offsets=torch.empty(case["experts"] + 1, dtype=torch.int32, device=DEV),
                     order=torch.empty(T * K, dtype=torch.int32, device=DEV), slots=torch.empty_like(ids))
        return state
    if case["kind"] == "sketch":
        N = T * K
        state.update(order=order, offsets=offsets, topk=K, bounds=bounds, most=int(np.diff(bounds).max()),
                     X=torch.randn(T, case["k"], generator=gen, device=DEV).to(dt),
                     dY=(torch.randn(N, case["d"], generator=gen, device=DEV) * 1e-3).to(dt),
                     S=torch.empty(case["experts"], case["d"], case["r"], device=DEV))
        if own:
            import rank_gradient_sketching_sketch_amd as L
            from rank_gradient_sketching_sketch_amd import binding as B

            state["m"] = L.MatrixDesc(case["d"], case["k"], case["r"], seed=SEED, step=STEP, matrix_id=FIRST_ID)
            n = L.logra_sketch_experts_workspace_bytes(state["m"], case["experts"], N,
                                                       B.LOGRA_BF16 if dt == torch.bfloat16 else B.LOGRA_F32)
            state["ws"] = torch.empty(max(16, n), dtype=torch.uint8, device=DEV)
        return state
    state.update(slots=slots, weights=weights, Ys=torch.randn(T * K, case["hidden"], generator=gen, device=DEV).to(dt))
    if case["kind"] == "combine":
        state["Y"] = torch.empty(T, case["hidden"], dtype=dt, device=DEV)
    else:
        state.update(dY=torch.randn(T, case["hidden"], generator=gen, device=DEV).to(dt),
                     dYs=torch.zeros(T * K, case["hidden"], dtype=dt, device=DEV), dw=torch.empty(T, K, device=DEV))
    return state


# --------------------------------------------------------------------- run --
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _run_own(kind, state)
    return {"clip": _clip, "dispatch": _dispatch, "combine": _combine, "combine_backward": _combine_backward,
            "sketch": _sketch}[kind](state)


def _run_own(kind, s):
    import rank_gradient_sketching_sketch_amd as L

    if kind == "clip":
        L.logra_grad_clip(s["list"], s["max_norm"], s["norm"], s["coef"], out=s["out_list"])
        return {"norm": s["norm"], "coef": s["coef"], "grads": s["out"]}
    if kind == "dispatch":
        L.logra_expert_sort(s["ids"], s["case"]["experts"], s["offsets"], s["order"], s["slots"])
        L.logra_expert_gather(s["X"], s["slots"], s["Xs"])
        return {"offsets": s["offsets"], "order": s["order"], "slots": s["slots"], "Xs": s["Xs"]}
    if kind == "combine":
        L.logra_expert_combine(s["Ys"], s["slots"], s["Y"], weights=s["weights"])
        return {"Y": s["Y"]}
    if kind == "combine_backward":
        L.logra_expert_combine_backward(s["dY"], s["Ys"], s["slots"], s["weights"], s["dYs"], s["dw"])
        return {"dYs": s["dYs"], "dw": s["dw"]}
    L.logra_sketch_experts(s["m"], s["offsets"], s["X"], s["dY"], s["S"], False, order=s["order"], topk=s["topk"],
                           ws=s["ws"])
    return {"S": s["S"]}


def _clip(s):
    f, d = s["flat"]["sketch"], s["flat"]["dense"]
    norm = torch.sqrt(f.double().square().sum() + d.double().square().sum())
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm)).float()
    return {"norm": norm.float().reshape(1), "coef": coef.reshape(1),
            "grads": {"sketch": f * coef, "dense": (d.float() * coef).to(d.dtype)}}


def _dispatch(s):
    ids, X, E = s["ids"].reshape(-1).long(), s["X"], s["case"]["experts"]
    K, n = s["ids"].shape[1], ids.numel()
    key = torch.where((ids < 0) | (ids >= E), E, ids)
    sorted_key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(sorted_key, torch.arange(E + 1, device=ids.device))
    place = torch.arange(n, device=ids.device)
    slots = torch.empty_like(order).scatter_(0, order, torch.where(sorted_key < E, place, -1))
    live = place < offsets[E]
    Xs = torch.where(live[:, None], X[order // K], torch.zeros((), dtype=X.dtype, device=X.device))
    return {"offsets": offsets.int(), "order": torch.where(live, order, -1).int(),
            "slots": slots.int().reshape(s["ids"].shape), "Xs": Xs}


def _rows(Ys, slots):
    """The experts' rows of every pair in 32 bits, zeros for dropped pairs: T x K x h."""
    got = Ys[slots.clamp(min=0).long()].float()
    return got * (slots >= 0)[..., None]


def _combine(s):
    return {"Y": (_rows(s["Ys"], s["slots"]) * s["weights"][..., None]).sum(1).to(s["Ys"].dtype)}


def _combine_backward(s):
    dY, slots, w = s["dY"].float(), s["slots"], s["weights"]
    dw = (_rows(s["Ys"], slots) * dY[:, None, :]).sum(-1)
    grads = (w[..., None] * dY[:, None, :]).reshape(-1, dY.shape[1]).to(s["dY"].dtype)
    flat = slots.reshape(-1).long()
    n = flat.numel()
    # dropped pairs write to a row behind the last
    dYs = torch.zeros(n + 1, dY.shape[1], dtype=grads.dtype, device=grads.device)
    dYs.index_copy_(0, torch.where(flat < 0, n, flat), grads)
    return {"dYs": dYs[:n], "dw": dw}


def _i64(x):
    return x - (1 << 64) if x >= (1 << 63) else x


def _shr(z, n):
    return (z >> n) & ((1 << (64 - n)) - 1)


def _finalize(z):
    z = (z ^ _shr(z, 30)) * _i64(MIX1)
    z = (z ^ _shr(z, 27)) * _i64(MIX2)
    return z ^ _shr(z, 31)


def _signs(case, device):
    """+-1 of every expert's sign matrix (E x r x k), from the counter hash in wrapping 64-bit integers."""
    E, r, k = case["experts"], case["r"], case["k"]
    g = _i64(GOLDEN)
    first = torch.tensor([SEED], device=device)
    key = _finalize((_finalize(first + g) ^ STEP) + g)
    key = _finalize((key ^ (FIRST_ID + torch.arange(E, device=device))) + g)
    row = torch.arange(r, device=device)[:, None] << 32
    word = torch.arange((k + 63) // 64, device=device)[None, :]
    words = _finalize(key[:, None, None] + ((row | word) + 1)[None] * g)
    bits = (words[..., None] >> torch.arange(64, device=device)) & 1
    return (1 - 2 * bits.to(torch.int8)).reshape(E, r, -1)[..., :k].float()


def _sketch(s):
    case, X, dY = s["case"], s["X"], s["dY"]
    counts = s["offsets"][1:] - s["offsets"][:-1]
    place = torch.arange(s["most"], device=X.device)
    live = place[None, :] < counts[:, None]                                  # E x (longest expert)
    slot = torch.where(live, s["offsets"][:-1, None] + place, 0).long()
    Xe = X[s["order"][slot].clamp(min=0).long() // s["topk"]].float() * live[..., None]
    dYe = dY[slot].float() * live[..., None]
    P = torch.bmm(Xe, _signs(case, X.device).transpose(1, 2).contiguous()) / math.sqrt(case["r"])
    return {"S": torch.bmm(dYe.transpose(1, 2).contiguous(), P)}


# -------------------------------------------------------------------- work --
def work(case):
    if case["kind"] == "clip":
        sketches, gains = _clip_shapes(case)
        n_s, n_g = sum(a * b for a, b in sketches), sum(a for a, in gains)
        return {"bytes": 2 * (4 * n_s + 2 * n_g) + 8, "flops": 3 * (n_s + n_g)}
    T, K, E = case["tokens"], min(case["topk"], case["experts"]), case["experts"]
    N, el = (T - case["pad"]) * K, 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "sketch":
        d, k, r = case["d"], case["k"], case["r"]
        used = min(E, N)
        return {"bytes": el * ((T - case["pad"]) * k + N * d) + 4 * E * d * r + 4 * (N + E + 1),
                "flops": 2 * N * r * (k + d) + used * r * k}
    h = case["hidden"]
    if case["kind"] == "dispatch":
        return {"bytes": el * h * ((T - case["pad"]) + N) + 4 * (3 * T * K + E + 1), "flops": N}
    if case["kind"] == "combine":
        return {"bytes": el * h * (T + N) + 8 * T * K, "flops": 2 * N * h}
    return {"bytes": el * h * ((T - case["pad"]) + 2 * N) + 12 * T * K, "flops": 3 * N * h}


# ------------------------------------------------------------------- exact --
def _mix64(z):
    z = (z ^ (z >> np.uint64(30))) * np.uint64(MIX1)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(MIX2)
    return z ^ (z >> np.uint64(31))


def _sign_rows(expert, r, k):
    """r x k signs of one expert, in unsigned 64-bit integers on the host."""
    with np.errstate(over="ignore"):
        g = np.uint64(GOLDEN)
        h = lambda x: _mix64(np.uint64(x) + g)  # noqa: E731
        key = h(h(h(np.array([SEED], np.uint64)) ^ np.uint64(STEP)) ^ np.uint64(FIRST_ID + expert))
        counter = (np.arange(r, dtype=np.uint64)[:, None] << np.uint64(32)) + np.arange((k + 63) // 64, dtype=np.uint64) + np.uint64(1)
        words = _mix64(key + counter * g)
    bits = np.unpackbits(words.view(np.uint8).reshape(r, -1), axis=1, bitorder="little")[:, :k]
    return torch.from_numpy(1.0 - 2.0 * bits).to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "clip":
        f, d = s["flat"]["sketch"], s["flat"]["dense"]
        norm = math.hypot(float(torch.linalg.vector_norm(f, dtype=torch.float64)),
                          float(torch.linalg.vector_norm(d, dtype=torch.float64)))
        coef = s["max_norm"] / norm if norm > s["max_norm"] else 1.0
        one = lambda v: torch.tensor([v], dtype=torch.float64, device=DEV)  # noqa: E731
        return {"norm": one(norm), "coef": one(coef), "grads": {"sketch": f.double() * coef, "dense": d.double() * coef}}
    if case["kind"] == "dispatch":
        ids, K, E = s["ids"].reshape(-1).long(), s["ids"].shape[1], case["experts"]
        Xs = torch.zeros(s["Xs"].shape, dtype=torch.float64, device=DEV)
        at, bounds = 0, [0]
        order, slots = torch.full_like(ids, -1), torch.full_like(ids, -1)
        for e in range(E):      # expert by expert, its pairs in their order
            pairs = (ids == e).nonzero().reshape(-1)
            n = pairs.numel()
            Xs[at:at + n] = s["X"][pairs // K].double()
            order[at:at + n] = pairs
            slots[pairs] = torch.arange(at, at + n, device=DEV)
            at += n
            bounds.append(at)
        return {"offsets": torch.tensor(bounds, device=DEV), "order": order, "slots": slots.reshape(s["ids"].shape), "Xs": Xs}
    if case["kind"] == "sketch":
        S = torch.zeros(s["S"].shape, dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            a, b = int(s["bounds"][e]), int(s["bounds"][e + 1])
            if a < b:
                G = s["dY"][a:b].double().T @ s["X"][s["order"][a:b].long() // s["topk"]].double()
                S[e] = G @ _sign_rows(e, case["r"], case["k"]).T / math.sqrt(case["r"])
        return {"S": S}
    slots, w = s["slots"], s["weights"].double()
    T, K = slots.shape
    if case["kind"] == "combine":
        Y = torch.zeros(T, case["hidden"], dtype=torch.float64, device=DEV)
        for j in range(K):      # one choice after the other
            t = (slots[:, j] >= 0).nonzero().reshape(-1)
            Y[t] += w[t, j, None] * s["Ys"][slots[t, j].long()].double()
        return {"Y": Y}
    dYs, dw = torch.zeros(s["dYs"].shape, dtype=torch.float64, device=DEV), torch.zeros(T, K, dtype=torch.float64, device=DEV)
    for j in range(K):
        t = (slots[:, j] >= 0).nonzero().reshape(-1)
        rows = slots[t, j].long()
        dYs[rows] = w[t, j, None] * s["dY"][t].double()
        dw[t, j] = torch.linalg.vecdot(s["dY"][t].double(), s["Ys"][rows].double())
    return {"dYs": dYs, "dw": dw}
