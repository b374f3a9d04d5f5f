"""The operators around a frozen int8 projection that is fine-tuned and served: low-rank adapters of many requests, layer
norm, and the AdamW step, as cases to be measured. `run` computes them in their plain form (elementary torch operations in
fp32) or, where `own` is set, through the package's entry points."""
import math

import torch

own = False

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 256          # values that share a scale of the 8-bit optimizer states
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.999, 1e-8, 0.01, 2e-4
LN_EPS = 1e-5


def listed():
    return [
        # one request generating one token through the 4096 x 4096 projection: latency alone
        dict(name="adapters_token", kind="adapters", dtype="bf16", T=1, S=1, n=8, K=4096, N=4096, R=16, spread="even"),
        # 64 requests generating one token each, 32 adapters in use, the gate projection of a 7B block
        dict(name="adapters_decode", kind="adapters", dtype="f16", T=64, S=64, n=32, K=4096, N=11008, R=16,
             spread="even"),
        # the prompts of 12 requests of very different lengths, some of them without an adapter
        dict(name="adapters_prefill", kind="adapters", dtype="bf16", T=4096, S=12, n=8, K=4096, N=4096, R=64,
             spread="ragged"),
        # fp32 with odd sizes and an odd rank: no row but the first starts on a 16-byte border
        dict(name="adapters_odd_grad", kind="adapters_grad", dtype="f32", T=777, S=5, n=3, K=1001, N=1530, R=6,
             spread="ragged"),
        # one training step of the up projection of a 7B block: two sequences of 2048 tokens, two adapters
        dict(name="adapters_grad", kind="adapters_grad", dtype="bf16", T=4096, S=2, n=2, K=4096, N=11008, R=16,
             spread="even"),
        # the same for the 70B widths, 16384 tokens of four tenants: the largest
        dict(name="adapters_grad_large", kind="adapters_grad", dtype="bf16", T=16384, S=16, n=4, K=8192, N=28672, R=32,
             spread="ragged"),
        # the norm of a decoding batch of eight
        dict(name="norm_token", kind="norm", dtype="f16", wdtype="f16", T=8, C=4096),
        # the norm in front of a 7B block's projections, 4096 tokens
        dict(name="norm", kind="norm", dtype="bf16", wdtype="f32", T=4096, C=4096),
        # its gradient, at the 70B width
        dict(name="norm_grad", kind="norm_grad", dtype="bf16", wdtype="f32", T=16384, C=8192),
        # biases and norm weights of a small model: a few short tensors
        dict(name="adamw_small", kind="adamw", dtype="f32", bits=32, master=False, sizes="4096*8,11008*4,31*3"),
        # all rank-16 adapters of a 7B model (32 blocks, seven projections), bf16 with fp32 masters, 8-bit states
        dict(name="adamw_adapters", kind="adamw", dtype="bf16", bits=8, master=True, sizes="65536*352,176128*96"),
        # the seven weights of a 7B block trained in full, 32-bit states
        dict(name="adamw_weights", kind="adamw", dtype="bf16", bits=32, master=False, sizes="16777216*4,45088768*3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer width: mostly a multiple of 64 or 8, sometimes any number."""
    n = _log(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(step, n // step * step)


def draw(rng):
    kind = rng.choice(("adapters", "adapters", "adapters_grad", "norm", "norm_grad", "adamw"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if kind in ("adapters", "adapters_grad"):
        K, N = _width(rng, 64, 11008), _width(rng, 64, 11008)
        R = rng.choice((4, 8, 16, 16, 32, 64, 128, rng.randint(1, 100)))
        if kind == "adapters" and rng.random() < 0.5:
            T = _log(rng, 1, 256)          # a decoding step: one token of each request
            S, n = T, _log(rng, 1, 64)
        else:
            T = _log(rng, 16, 8192)
            S, n = _log(rng, 1, min(T, 64)), _log(rng, 1, 16)
        return dict(kind=kind, dtype=dtype, T=T, S=S, n=n, K=K, N=N, R=R, spread=rng.choice(("even", "ragged")))
    if kind in ("norm", "norm_grad"):
        C = _width(rng, 64, 16384)
        T = _log(rng, 1, min(16384, (1 << 27) // C))
        return dict(kind=kind, dtype=dtype, wdtype=rng.choice((dtype, "f32")), T=T, C=C)
    groups, left = [], _log(rng, 1000, 100_000_000)
    for _ in range(rng.randint(1, 4)):
        n = max(1, min(_log(rng, 1, 1 << 24), left))
        count = max(1, min(rng.randint(1, 100), left // n))
        groups.append("%d*%d" % (n, count))
        left = max(1, left - n * count)
    return dict(kind="adamw", dtype=dtype, bits=rng.choice((8, 32)), master=dtype != "f32" and rng.random() < 0.5,
                sizes=",".join(groups))


def _sizes(case):
    out = []
    for part in case["sizes"].split(","):
        n, count = part.split("*")
        out += [int(n)] * int(count)
    return out


def _segments(case, seed):
    """Lengths of the requests and their adapters, on the host: even or very uneven lengths (some empty), one in eight
    requests of a ragged batch without an adapter."""
    g = torch.Generator().manual_seed(seed)
    T, S, n = case["T"], case["S"], case["n"]
    if case["spread"] == "even":
        off = torch.arange(S + 1) * T // S
        ids = torch.randperm(max(S, n), generator=g)[:S] % n
    else:
        cut = (torch.rand(S - 1, generator=g, dtype=torch.float64) ** 2 * (T + 1)).long().clamp(0, T)
        off = torch.cat([torch.tensor([0]), cut.sort().values, torch.tensor([T])])
        ids = torch.randint(0, n, (S,), generator=g)
        ids[torch.rand(S, generator=g) < 0.125] = -1
    return off, ids


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _activations(g, T, C, dtype):
    """N(0, 1) with one feature in a thousand 20 times as large, as the inputs of such layers have."""
    x = torch.randn((T, C), generator=g, device=DEV)
    cols = torch.randperm(C, generator=g, device=DEV)[: max(1, C // 1000)]
    x[:, cols] *= 20
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = DT[case["dtype"]]
    s = dict(case)
    if case["kind"] in ("adapters", "adapters_grad"):
        T, n, K, N, R = (case[k] for k in ("T", "n", "K", "N", "R"))
        off, ids = _segments(case, seed)
        s["off"], s["ids"] = off.to(DEV, torch.int32), ids.to(DEV, torch.int32)
        s["X"] = _activations(g, T, K, dt)
        s["A"] = _normal(g, (n, R, K), dt, K ** -0.5)
        s["B"] = _normal(g, (n, N, R), dt, 0.02)
        s["scaling"] = torch.rand(n, generator=g, device=DEV) + 0.5
        if case["kind"] == "adapters":
            s["base"] = _normal(g, (T, N), dt)
        else:
            s["G"] = _normal(g, (T, N), dt, 0.01)
            s["base"] = _normal(g, (T, K), dt, 0.01)
            s["V"] = _shrink(s)            # kept by the forward pass
    elif case["kind"] in ("norm", "norm_grad"):
        T, C, wt = case["T"], case["C"], DT[case["wdtype"]]
        s["X"] = (_activations(g, T, C, torch.float32) + 0.3).to(dt)
        s["w"] = (1 + 0.1 * torch.randn(C, generator=g, device=DEV)).to(wt)
        s["b"] = _normal(g, (C,), wt, 0.1)
        if case["kind"] == "norm_grad":
            s["G"] = _normal(g, (T, C), dt, 0.01)
            s["mean"], s["rstd"] = _norm_stats(s["X"])
    else:
        sizes = _sizes(case)
        at = [0]
        for n in sizes:
            at.append(at[-1] + -(-n // BLOCK) * BLOCK)
        total = at[-1]
        real = torch.ones(total, device=DEV)
        for n, a, b in zip(sizes, at, at[1:]):
            if a + n < b:
                real[a + n:b] = 0          # between tensors: zeros, which stay zeros
        def new(scale):
            return torch.randn(total, generator=g, device=DEV).mul_(scale).mul_(real)
        w = new(0.02)
        s["P"] = w.to(dt)
        s["W"] = w if case["master"] else None
        s["G"] = new(1e-3).to(dt)
        m = new(3e-4)
        q = torch.randn(total, generator=g, device=DEV).exp_().mul_(1e-3).mul_(real)
        if case["bits"] == 8:
            s["M"], s["Ms"] = _to_8bit(m)
            s["Q"], s["Qs"] = _to_8bit(q)
        else:
            s["M"], s["V"] = m, q.square_()
        s["scale"] = torch.rand(1, generator=g, device=DEV) * 0.5 + 0.5      # what clipping multiplies gradients with
        s["step"] = 10
        s["at"], s["sizes"] = at, sizes
        if own:
            import int8_quantized_linear_rowwise_amd as I8

            def cut(x, per=1):
                return [x[a // per: a // per + -(-n // per)] for n, a in zip(sizes, at)]
            s["opt"] = I8.AdamWPlan(
                cut(s["P"]), cut(s["G"]), cut(s["M"]), cut(s["Q" if case["bits"] == 8 else "V"]),
                m_scale=cut(s["Ms"], BLOCK) if case["bits"] == 8 else None,
                v_scale=cut(s["Qs"], BLOCK) if case["bits"] == 8 else None,
                master=cut(s["W"]) if case["master"] else None)
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------------


def _token_adapters(s):
    """The adapter of each token, and where it is one: from the segments, by comparison."""
    t = torch.arange(s["T"], device=DEV, dtype=torch.int32)
    seg = (t[:, None] >= s["off"][None, 1:-1]).sum(1)
    a = s["ids"][seg]
    return a, (a >= 0) & (a < s["n"])


def _own_columns(v, s):
    """v: T x (n R), every token's products with every adapter; those with its own, others 0."""
    a, has = _token_adapters(s)
    mine = (torch.arange(s["n"], device=DEV)[None] == a[:, None]) & has[:, None]
    return torch.where(mine[:, :, None], v.view(-1, s["n"], s["R"]), 0.0).view(v.shape)


def _shrink(s):
    v = s["X"].float() @ s["A"].float().view(-1, s["K"]).t()
    return _own_columns(v, s).view(-1, s["n"], s["R"]).sum(1)


def _adapters(s):
    v = _own_columns(s["X"].float() @ s["A"].float().view(-1, s["K"]).t(), s)
    v = v * s["scaling"].repeat_interleave(s["R"], output_size=v.shape[1])
    b = s["B"].float().transpose(1, 2).reshape(-1, s["N"])
    return (s["base"].float() + v @ b).to(s["X"].dtype)


def _adapters_grad(s):
    G, X, n, R = s["G"].float(), s["X"].float(), s["n"], s["R"]
    a = s["A"].float().view(n * R, -1)
    b = s["B"].float().transpose(1, 2).reshape(n * R, -1)
    scaling = s["scaling"].repeat_interleave(R, output_size=n * R)
    dv = _own_columns(G @ b.t(), s) * scaling
    gx = s["base"].float() + dv @ a
    v = _own_columns(s["V"].repeat(1, n), s) * scaling
    ga = (dv.t() @ X).view(n, R, -1)
    gb = (v.t() @ G).view(n, R, -1).transpose(1, 2).contiguous()
    dt = s["X"].dtype
    return gx.to(dt), ga.to(dt), gb.to(dt)


def _norm_stats(x):
    x = x.float()
    mean = x.mean(1)
    return mean, 1.0 / torch.sqrt((x - mean[:, None]).square().mean(1) + LN_EPS)


def _norm(s):
    mean, rstd = _norm_stats(s["X"])
    h = (s["X"].float() - mean[:, None]) * rstd[:, None]
    return (h * s["w"].float() + s["b"].float()).to(s["X"].dtype), mean, rstd


def _norm_grad(s):
    g = s["G"].float()
    h = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    u = g * s["w"].float()
    gx = s["rstd"][:, None] * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
    return gx.to(s["X"].dtype), (g * h).sum(0).to(s["w"].dtype), g.sum(0).to(s["w"].dtype)


def _to_8bit(x, positive=False):
    """Blocks of 256 values as e4m3 times the least power of two (from 2^-126) that keeps the block within 448; with
    `positive`, what is over 0 stays over 0."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1)
    f, e = torch.frexp(top)                # top = f 2^e, 0.5 <= f < 1
    e = torch.where(f > 0.875, e - 8, e - 9).clamp(min=-126)
    scale = ((e + 127) << 23).view(torch.float32)
    y = x * (((127 - e) << 23).view(torch.float32))[:, None]
    if positive:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn).view(-1), scale


def _from_8bit(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw(s):
    t = s["step"]
    low = s["bits"] == 8
    g = s["G"].float() * s["scale"]
    m = _from_8bit(s["M"], s["Ms"]) if low else s["M"]
    v = _from_8bit(s["Q"], s["Qs"]).square() if low else s["V"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    q = torch.sqrt(v)
    w = s["W"] if s["master"] else s["P"].float()
    w = w * (1 - LR * DECAY) - m / (q * (1 / math.sqrt(1 - BETA2 ** t)) + EPS) * (LR / (1 - BETA1 ** t))
    s["P"].copy_(w)
    if s["master"]:
        s["W"].copy_(w)
    if low:
        code, scale = _to_8bit(m)
        s["M"].copy_(code), s["Ms"].copy_(scale)
        code, scale = _to_8bit(q, positive=True)
        s["Q"].copy_(code), s["Qs"].copy_(scale)
    else:
        s["M"].copy_(m), s["V"].copy_(v)


# ---- one pass -------------------------------------------------------------------------------------------------------


def _states(s):
    names = ("P", "W", "M", "Ms", "Q", "Qs") if s["bits"] == 8 else ("P", "W", "M", "V")
    return {k: s[k] for k in names if s[k] is not None}


def run(s):
    kind = s["kind"]
    if kind == "adamw":
        s["step"] += 1
        if own:
            s["opt"].step(s["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, grad_scale=s["scale"])
        else:
            _adamw(s)
        return _states(s)
    if not own:
        return {"adapters": _adapters, "adapters_grad": _adapters_grad, "norm": _norm, "norm_grad": _norm_grad}[kind](s)
    import int8_quantized_linear_rowwise_amd as I8
    if kind == "adapters":
        return I8.lora_forward(s["X"], s["A"], s["B"], s["scaling"], s["off"], s["ids"], base=s["base"])
    if kind == "adapters_grad":
        return I8.lora_backward(s["G"], s["X"], s["V"], s["A"], s["B"], s["scaling"], s["off"], s["ids"],
                                base_grad=s["base"])
    if kind == "norm":
        return I8.layer_norm_forward(s["X"], s["w"], s["b"], eps=LN_EPS)
    return I8.layer_norm_backward(s["G"], s["X"], s["mean"], s["rstd"], s["w"])


def work(case):
    kind, e = case["kind"], SIZE[case["dtype"]]
    if kind in ("adapters", "adapters_grad"):
        T, S, n, K, N, R = (case[k] for k in ("T", "S", "n", "K", "N", "R"))
        used = min(S, n)
        if kind == "adapters":
            return dict(bytes=T * (K + 2 * N) * e + used * (K + N) * R * e, flops=2 * T * R * (K + N))
        return dict(bytes=T * (N + 3 * K) * e + 4 * T * R + (used + n) * (K + N) * R * e, flops=4 * T * R * (K + N))
    if kind in ("norm", "norm_grad"):
        T, C, we = case["T"], case["C"], SIZE[case["wdtype"]]
        if kind == "norm":
            return dict(bytes=2 * T * C * e + 2 * C * we + 8 * T, flops=8 * T * C)
        return dict(bytes=3 * T * C * e + 3 * C * we + 8 * T, flops=14 * T * C)
    n = sum(_sizes(case))
    per = (3 * e + 8 * case["master"] - e * case["master"]) + (4 if case["bits"] == 8 else 16)
    return dict(bytes=n * per, flops=16 * n)


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------


def _exact_8bit(x, positive):
    out, scales = torch.empty_like(x), torch.empty(x.numel() // BLOCK, dtype=torch.float64, device=DEV)
    for i in range(0, x.numel(), 1 << 24):
        b = x[i:i + (1 << 24)].view(-1, BLOCK)
        top = b.abs().max(1).values
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448.0))
        e = torch.where(top * torch.pow(2.0, -e) > 448.0, e + 1, e)
        e = torch.where(top > 0, e, -126.0).clamp(min=-126.0)
        unit = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV), e)
        y = b / unit[:, None]
        if positive:
            y = torch.where(b > 0, torch.maximum(y, torch.tensor(2.0 ** -9, dtype=torch.float64, device=DEV)), y)
        mag = y.abs()
        step = torch.pow(2.0, torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)      # e4m3's spacing there
        out[i:i + (1 << 24)] = (torch.sign(y) * torch.round(mag / step) * step).view(-1)
        scales[i // BLOCK: i // BLOCK + unit.numel()] = unit
    return out, scales


def exact(case, seed):
    s = prepare(case, seed)
    kind, d = case["kind"], torch.float64
    if kind in ("adapters", "adapters_grad"):
        off, ids = s["off"].tolist(), s["ids"].tolist()
        A, B, sc, X = s["A"].to(d), s["B"].to(d), s["scaling"].to(d), s["X"].to(d)
        Y = s["base"].to(d)
        if kind == "adapters":
            for lo, hi, a in zip(off, off[1:], ids):
                if a >= 0 and hi > lo:
                    Y[lo:hi] += sc[a] * ((X[lo:hi] @ A[a].t()) @ B[a].t())
            return Y
        gA, gB, G = torch.zeros_like(A), torch.zeros_like(B), s["G"].to(d)
        for lo, hi, a in zip(off, off[1:], ids):
            if a >= 0 and hi > lo:
                dv = sc[a] * (G[lo:hi] @ B[a])
                Y[lo:hi] += dv @ A[a]
                gA[a] += dv.t() @ X[lo:hi]
                gB[a] += sc[a] * (G[lo:hi].t() @ (X[lo:hi] @ A[a].t()))
        return Y, gA, gB
    if kind in ("norm", "norm_grad"):
        X, w = s["X"].to(d), s["w"].to(d)
        mean = X.sum(1, keepdim=True) / case["C"]
        rstd = (((X - mean) ** 2).sum(1, keepdim=True) / case["C"] + LN_EPS) ** -0.5
        h = (X - mean) * rstd
        if kind == "norm":
            return h * w + s["b"].to(d), mean[:, 0], rstd[:, 0]
        G = s["G"].to(d)
        u = G * w
        gx = rstd * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
        return gx, (G * h).sum(0), G.sum(0)
    t = s["step"] + 1
    g = s["G"].to(d) * s["scale"].to(d)
    low = case["bits"] == 8
    m, v = s["M"].to(d), s["Q" if low else "V"].to(d)
    if low:
        m = (m.view(-1, BLOCK) * s["Ms"].to(d)[:, None]).view(-1)
        v = (v.view(-1, BLOCK) * s["Qs"].to(d)[:, None]).view(-1) ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    w = (s["W"] if case["master"] else s["P"]).to(d)
    w = w - LR * (DECAY * w + (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS))
    out = {"P": w}
    if case["master"]:
        out["W"] = w
    if low:
        out["M"], out["Ms"] = _exact_8bit(m, False)
        out["Q"], out["Qs"] = _exact_8bit(torch.sqrt(v), True)
    else:
        out["M"], out["V"] = m, v
    return out
