"""The operators of a mixture of experts whose projections are frozen in int8, as cases to be measured: the sort of
tokens by expert, the products of each expert with its rows and their input gradient, the weighted sum of each token's
rows with its gradient, and the norm of all gradients with the clipping of what the optimizer reads. `run` computes them
in their plain form (elementary torch operations in fp32) or, where `own` is set, through the package's entry points."""
import math

import torch

own = False

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
TAU = 6.0            # a feature column with a larger value is an outlier column
BLOCK = 256          # tensors of a gradient list start on multiples of this many values
SHRINK = 0.999       # max_norm of a pass against the one before: gradients clipped in place have to be clipped again
LARGEST = 4096 * 2 * 4096 * 11008      # multiply-adds of the largest listed product


def listed():
    return [
        # one token of one request and its two experts of eight: latency alone
        dict(name="sort_token", kind="sort", T=1, k=2, E=8, drop=False, ids="int64"),
        # a batch of 16384 tokens, eight experts each of 128
        dict(name="sort", kind="sort", T=16384, k=8, E=128, drop=False, ids="int64"),
        # one token through its two experts, 7B block widths: the weights of two experts, read once
        dict(name="experts_token", kind="experts", dtype="bf16", T=1, k=2, E=8, K=4096, N=11008, drop=False),
        # 64 requests generating one token each, four narrow experts of 64
        dict(name="experts_decode", kind="experts", dtype="f16", T=64, k=4, E=64, K=2048, N=1408, drop=False),
        # prompts of 4096 tokens, two experts of eight each
        dict(name="experts_prefill", kind="experts", dtype="bf16", T=4096, k=2, E=8, K=4096, N=11008, drop=False),
        # fp32 with odd widths: no row but the first starts on a 16-byte border; some choices over an expert's capacity
        dict(name="experts_odd", kind="experts", dtype="f32", T=777, k=3, E=5, K=1001, N=1530, drop=True),
        # input gradient of the prompts' products
        dict(name="experts_grad", kind="experts_grad", dtype="bf16", T=4096, k=2, E=8, K=4096, N=11008, drop=False),
        # the same of many narrow experts with uneven numbers of rows
        dict(name="experts_grad_narrow", kind="experts_grad", dtype="f16", T=4096, k=4, E=64, K=2048, N=1408,
             drop=True),
        # back from the experts' rows to 4096 tokens, added to the residual
        dict(name="combine", kind="combine", dtype="bf16", T=4096, k=2, E=8, N=4096, drop=False),
        # the gradients of the rows and of the weights, eight experts for each of 8192 tokens
        dict(name="combine_grad", kind="combine_grad", dtype="bf16", T=8192, k=8, E=64, N=2048, drop=True),
        # gradients of all rank-16 adapters of a 7B model (32 blocks, seven projections), clipped in place
        dict(name="clip_adapters", kind="clip", dtype="bf16", sizes="65536*352,176128*96"),
        # gradients of the seven weights of a 7B block: the factor that the optimizer's step multiplies them with
        dict(name="norm_weights", kind="norm", dtype="bf16", sizes="16777216*4,45088768*3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer width: mostly a multiple of 64 or 8, sometimes any number."""
    n = _log(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(step, n // step * step)


def draw(rng):
    kind = rng.choice(("sort", "experts", "experts", "experts", "experts_grad", "experts_grad", "combine",
                       "combine_grad", "clip", "norm"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if kind in ("clip", "norm"):
        groups, left = [], _log(rng, 1000, 100_000_000)
        for _ in range(rng.randint(1, 4)):
            n = max(1, min(_log(rng, 1, 1 << 24), left))
            count = max(1, min(rng.randint(1, 100), left // n))
            groups.append("%d*%d" % (n, count))
            left = max(1, left - n * count)
        return dict(kind=kind, dtype=dtype, sizes=",".join(groups))
    E = _log(rng, 1, 128)
    k = min(E, rng.randint(1, 8))
    drop = rng.random() < 0.3
    if kind == "sort":
        return dict(kind=kind, T=_log(rng, 1, 16384), k=k, E=E, drop=drop, ids=rng.choice(("int32", "int64")))
    N = _width(rng, 64, 11008)
    if kind in ("combine", "combine_grad"):
        T = _log(rng, 1, max(1, min(8192, (1 << 27) // (k * N))))
        return dict(kind=kind, dtype=dtype, T=T, k=k, E=E, N=N, drop=drop)
    K = _width(rng, 64, 4096)
    E = max(1, min(E, (1 << 29) // (K * N)))
    k = min(k, E)
    top = max(1, min(8192, LARGEST // 4 // (k * K * N)))
    T = _log(rng, 1, min(256, top)) if kind == "experts" and rng.random() < 0.5 else _log(rng, 1, top)
    return dict(kind=kind, dtype=dtype, T=T, k=k, E=E, K=K, N=N, drop=drop)


# ---- inputs ---------------------------------------------------------------------------------------------------------


def _sizes(case):
    out = []
    for part in case["sizes"].split(","):
        n, count = part.split("*")
        out += [int(n)] * int(count)
    return out


def _choose(g, case):
    """The experts of each token, best first: a score that some experts win more often than others. With `drop`, one
    choice in sixteen is -1 (over the expert's capacity)."""
    T, k, E = case["T"], case["k"], case["E"]
    score = torch.randn((T, E), generator=g, device=DEV) + 0.7 * torch.randn(E, generator=g, device=DEV)
    ids = score.topk(k, 1).indices
    if case["drop"]:
        ids[torch.rand((T, k), generator=g, device=DEV) < 1 / 16] = -1
    return ids


def _sorted(ids, E):
    """Offsets of the experts' rows, the token of each row (-1 behind the last), the row of each choice (-1: none)."""
    flat = ids.reshape(-1).long()
    R = flat.numel()
    routed = (flat >= 0) & (flat < E)
    key = torch.where(routed, flat, E)
    by, order = key.sort(stable=True)
    off = torch.searchsorted(by, torch.arange(E + 1, device=DEV))
    at = torch.arange(R, device=DEV)
    row = torch.empty_like(order)
    row[order] = at
    token = torch.where(at < off[-1], order // ids.shape[1], -1)
    position = torch.where(routed, row, -1).view(ids.shape)
    return off.int(), token.int(), position.int()


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _activations(g, T, C, dtype):
    """N(0, 1) with one feature in a thousand 20 times as large, as the inputs of such layers have."""
    x = torch.randn((T, C), generator=g, device=DEV)
    cols = torch.randperm(C, generator=g, device=DEV)[: max(1, C // 1000)]
    x[:, cols] *= 20
    return x.to(dtype)


def _weights(g, E, N, K):
    """Every expert's weight in int8, a scale for each output feature."""
    CB = torch.empty((E, N, K), dtype=torch.int8, device=DEV)
    SCB = torch.empty((E, N), device=DEV)
    for e in range(E):
        w = (torch.randn((N, K), generator=g, device=DEV) * K ** -0.5).half().float()
        s = w.abs().amax(1)
        SCB[e] = s
        CB[e] = torch.round(w * (127.0 / s)[:, None]).to(torch.int8)
    return CB, SCB


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    kind = case["kind"]
    if kind in ("clip", "norm"):
        sizes = _sizes(case)
        at = [0]
        for n in sizes:
            at.append(at[-1] + -(-n // BLOCK) * BLOCK)
        G = torch.randn(at[-1], generator=g, device=DEV).mul_(1e-3)
        for n, a, b in zip(sizes, at, at[1:]):
            if a + n < b:
                G[a + n:b] = 0             # between tensors: zeros, which change no norm
        s["G"] = G.to(DT[case["dtype"]])
        s["max_norm"] = 5e-4 * sum(sizes) ** 0.5                 # half of the norm before scaling
        if kind == "norm":
            s["scale"] = torch.rand(1, generator=g, device=DEV) * 0.5 + 0.5      # what undoes the loss's scale
        if own:
            import int8_quantized_linear_rowwise_amd as I8
            s["plan"] = I8.GradNormPlan([s["G"][a:a + n] for n, a in zip(sizes, at)])
        return s
    ids = _choose(g, case)
    if kind == "sort":
        s["ids"] = ids.to(getattr(torch, case["ids"]))
        return s
    dt, T, k, E, N = DT[case["dtype"]], case["T"], case["k"], case["E"], case["N"]
    s["off"], s["token"], s["position"] = _sorted(ids, E)
    s["bounds"] = s["off"].tolist()
    if kind in ("experts", "experts_grad"):
        K = case["K"]
        s["CB"], s["SCB"] = _weights(g, E, N, K)
        if kind == "experts":
            s["X"] = _activations(g, T, K, dt)
        else:
            s["G"] = _normal(g, (T * k, N), dt, 0.01)
        return s
    s["Y"] = _normal(g, (T * k, N), dt)
    s["gate"] = torch.rand((T, k), generator=g, device=DEV).softmax(1)
    if kind == "combine":
        s["base"] = _normal(g, (T, N), dt)
    else:
        s["G"] = _normal(g, (T, N), dt, 0.01)
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------------


def _segments(s):
    """Expert, first row and end of every expert with rows, from the host's copy of the offsets."""
    b = s["bounds"]
    return [(e, lo, hi) for e, (lo, hi) in enumerate(zip(b, b[1:])) if hi > lo]


def _dequantized(s, e):
    return (s["CB"][e].float() * (s["SCB"][e] * (1.0 / 127.0))[:, None]).half()


def _experts(s):
    x16 = s["X"].half().float()
    mag = x16.abs()
    out_cols = (mag > TAU).any(0)
    top = torch.where(out_cols, 0.0, mag).amax(1)
    inv = torch.where(top > 0, torch.div(torch.full_like(top, 127.0), top), 0.0)      # one rounding, not two
    codes = torch.where(out_cols, 0.0, torch.round(x16 * inv[:, None]))
    O = out_cols.nonzero()[:, 0]
    sub = x16[:, O]
    y = torch.zeros((s["T"] * s["k"], s["N"]), device=DEV)
    for e, lo, hi in _segments(s):
        t = s["token"][lo:hi].long()
        y[lo:hi] = (codes[t] @ s["CB"][e].float().t()) * top[t][:, None] * (s["SCB"][e] * (1.0 / 16129.0))
        y[lo:hi] += sub[t] @ _dequantized(s, e)[:, O].float().t()
    return y.to(s["X"].dtype)


def _experts_grad(s):
    gx = torch.zeros((s["T"] * s["k"], s["K"]), device=DEV)
    for e, lo, hi in _segments(s):
        gx[lo:hi] = s["G"][lo:hi].half().float() @ _dequantized(s, e).float()
    return gx.to(s["G"].dtype)


def _combine(s):
    has = s["position"] >= 0
    y = s["base"].float()
    for j in range(s["k"]):
        w = torch.where(has[:, j], s["gate"][:, j], 0.0)
        y = y + w[:, None] * s["Y"][s["position"][:, j].clamp(min=0).long()].float()
    return y.to(s["base"].dtype)


def _combine_grad(s):
    G, has = s["G"].float(), s["position"] >= 0
    token = s["token"].clamp(min=0).long()
    gate = torch.zeros(s["T"] * s["k"] + 1, device=DEV)
    gate[torch.where(has, s["position"], s["T"] * s["k"]).long()] = s["gate"]
    gy = torch.where(s["token"] >= 0, gate[:-1], 0.0)[:, None] * G[token]
    dots = [(G * s["Y"][s["position"][:, j].clamp(min=0).long()].float()).sum(1) for j in range(s["k"])]
    return gy.to(s["G"].dtype), torch.where(has, torch.stack(dots, 1), 0.0)


def _norm(s):
    scale = s["scale"].double()[0] if s["kind"] == "norm" else 1.0
    norm = s["G"].float().square().sum(dtype=torch.float64).sqrt() * scale
    factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0) * scale
    return norm.float(), factor.float(), (~torch.isfinite(norm)).float()


# ---- one pass -------------------------------------------------------------------------------------------------------


def run(s):
    kind = s["kind"]
    if kind == "clip":
        s["max_norm"] *= SHRINK
    if not own:
        if kind == "sort":
            return _sorted(s["ids"], s["E"])
        if kind in ("clip", "norm"):
            norm, factor, bad = _norm(s)
            if kind == "norm":
                return norm, factor, bad
            s["G"].copy_(s["G"].float() * factor)
            return s["G"], norm, factor, bad
        return {"experts": _experts, "experts_grad": _experts_grad, "combine": _combine,
                "combine_grad": _combine_grad}[kind](s)
    import int8_quantized_linear_rowwise_amd as I8
    if kind == "sort":
        return I8.expert_sort(s["ids"], s["E"])
    if kind == "experts":
        return I8.expert_forward(s["X"], s["CB"], s["SCB"], s["off"], rows=s["token"], threshold=TAU)
    if kind == "experts_grad":
        return I8.expert_backward(s["G"], s["CB"], s["SCB"], s["off"])
    if kind == "combine":
        return I8.expert_combine(s["Y"], s["position"], s["gate"], base=s["base"])
    if kind == "combine_grad":
        return I8.expert_combine_backward(s["G"], s["position"], s["gate"], s["Y"], n_rows=s["off"][-1:])
    if kind == "norm":
        return s["plan"].norm(s["max_norm"], grad_scale=s["scale"])
    return (s["G"], *s["plan"].clip(s["max_norm"]))


def work(case):
    kind = case["kind"]
    if kind in ("clip", "norm"):
        n, e = sum(_sizes(case)), SIZE[case["dtype"]]
        return dict(bytes=n * e * (2 if kind == "clip" else 1), flops=n * (3 if kind == "clip" else 2))
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    if kind == "sort":
        return dict(bytes=R * ((8 if case["ids"] == "int64" else 4) + 8) + 4 * E, flops=2 * R)
    e, N = SIZE[case["dtype"]], case["N"]
    if kind in ("experts", "experts_grad"):
        K, used = case["K"], min(E, R)
        rows = (T * K + R * N) * e if kind == "experts" else R * (K + N) * e
        return dict(bytes=rows + used * N * (K + 4) + 4 * R, flops=2 * R * N * K)
    if kind == "combine":
        return dict(bytes=(R + 2 * T) * N * e + 8 * R, flops=2 * R * N)
    return dict(bytes=(2 * R + T) * N * e + 12 * R, flops=3 * R * N)


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------


def _exact_sort(ids, E):
    flat = ids.reshape(-1).tolist()
    k = ids.shape[1]
    lists = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(i)
    off, token, position = [0], [], [-1] * len(flat)
    for mine in lists:
        for i in mine:
            position[i] = len(token)
            token.append(i // k)
        off.append(len(token))
    token += [-1] * (len(flat) - len(token))

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    return ints(off), ints(token), ints(position).view(ids.shape)


def _exact_codes(X):
    """Codes, scales and outlier columns: fp16 values, divided by their row's largest over 127, the quotient and the
    product each rounded to fp32 as the definition says."""
    d = torch.float64
    x = X.to(torch.float16).to(d)
    cols = (x.abs() > TAU).any(dim=0)
    inner = x * (~cols).to(d)
    top = inner.abs().max(dim=1).values
    inv = torch.div(torch.full_like(top, 127.0), torch.where(top > 0, top, 1.0)).float().to(d)
    codes = torch.round((inner * inv[:, None]).float().to(d))
    return torch.where((top > 0)[:, None], codes, 0.0), top, x * cols.to(d)


def _exact_weight(cb, scb):
    unit = (scb.double() * torch.tensor(1 / 127, dtype=torch.float32).double().item()).float().double()
    return (cb.double() * unit[:, None]).float().half().double()


def exact(case, seed):
    s = prepare(case, seed)
    kind, d = case["kind"], torch.float64
    if kind in ("clip", "norm"):
        max_norm = s["max_norm"] * (SHRINK if kind == "clip" else 1.0)
        total = sum(s["G"][i:i + (1 << 26)].to(d).pow(2).sum() for i in range(0, s["G"].numel(), 1 << 26))
        c = s["scale"].to(d)[0] if kind == "norm" else torch.ones((), dtype=d, device=DEV)
        norm = c * total.sqrt()
        factor = c * torch.minimum(max_norm / (norm + 1e-6), torch.ones_like(norm))
        out = norm, factor, torch.zeros_like(norm)
        return out if kind == "norm" else (s["G"].to(d) * factor, *out)
    if kind == "sort":
        return _exact_sort(s["ids"], case["E"])
    off, R, N = s["off"].tolist(), case["T"] * case["k"], case["N"]
    token = s["token"].long()
    if kind == "experts":
        codes, top, outliers = _exact_codes(s["X"])
        Y = torch.zeros((R, N), dtype=d, device=DEV)
        for e in range(case["E"]):
            t = token[off[e]:off[e + 1]]
            if t.numel():
                w = s["CB"][e].to(d) * (s["SCB"][e].to(d) / 127 ** 2)[:, None]
                Y[off[e]:off[e + 1]] = top[t, None] * (codes[t] @ w.t()) \
                    + outliers[t] @ _exact_weight(s["CB"][e], s["SCB"][e]).t()
        return Y
    if kind == "experts_grad":
        gx = torch.zeros((R, case["K"]), dtype=d, device=DEV)
        for e in range(case["E"]):
            if off[e + 1] > off[e]:
                gx[off[e]:off[e + 1]] = s["G"][off[e]:off[e + 1]].to(torch.float16).to(d) \
                    @ _exact_weight(s["CB"][e], s["SCB"][e])
        return gx
    live = torch.arange(R, device=DEV) < off[-1]
    t, j = (s["position"] >= 0).nonzero(as_tuple=True)
    row = s["position"][t, j].long()
    w = torch.zeros(R, dtype=d, device=DEV)
    w[row] = s["gate"][t, j].to(d)
    if kind == "combine":
        return s["base"].to(d).index_add(0, t, w[row, None] * s["Y"][row].to(d))
    gy = w[:, None] * s["G"][token.clamp(min=0)].to(d) * live[:, None]
    gg = torch.zeros((case["T"], case["k"]), dtype=d, device=DEV)
    gg[t, j] = (s["G"][t].to(d) * s["Y"][row].to(d)).sum(1)
    return gy, gg
