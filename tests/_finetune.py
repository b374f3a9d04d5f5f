"""Plain 64-bit forms of the operators around the frozen projection (adapters,
layer norm, AdamW) with the error each result may have, and input makers.

Error bounds count roundings: `u` = 2^-24 is half a step of fp32 relative to
the value, eps / 2 that of the output type. A sum of n products in fp32, in
any order, is off by at most n u times the sum of the magnitudes (first
order; 1 % is added for the higher orders). V and dV enter products with
16-bit operands as the sum of two 16-bit values: at most 2^-17 relative.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
D = torch.float64
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}      # half a step of fp16's denormals


def half_step(dt: str) -> float:
    return torch.finfo(DT[dt]).eps / 2


def randn(shape, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dt])


def assert_within(got, want, lim, what):
    got, want, lim = got.detach().to("cpu", D), want.to("cpu", D), lim.to("cpu", D)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.numel() == 0:
        return
    err = (got - want).abs()
    bad = ~(err <= lim)
    if bad.any():
        i = int(torch.where(bad.view(-1), (err / lim.clamp(min=1e-300)).view(-1).nan_to_num(1e30, 1e30), 0.0).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} beyond their bound; worst at flat {i}: got "
                             f"{got.view(-1)[i].item()!r}, want {want.view(-1)[i].item()!r}, bound "
                             f"{lim.view(-1)[i].item():.3g}")


# ---- adapters


def lora_inputs(dt, T, K, N, R, n, seed):
    X = randn((T, K), dt, seed)
    if K > 1:
        X[:, seed % K] *= 20
    return dict(X=X, A=randn((n, R, K), dt, seed + 1, K ** -0.5), B=randn((n, N, R), dt, seed + 2, 0.3),
                scaling=torch.rand(n, generator=torch.Generator().manual_seed(seed + 3)) + 0.5,
                base=randn((T, N), dt, seed + 4), G=randn((T, N), dt, seed + 5, 0.1),
                base_grad=randn((T, K), dt, seed + 6, 0.1))


def segments_of(off, ids, n, T):
    """(first row, last row + 1, adapter or -1) of every segment; offsets None: one segment."""
    off = [0, T] if off is None else list(off)
    if len(off) > 1:
        off[0], off[-1] = 0, T
    ids = list(range(len(off) - 1)) if ids is None else list(ids)
    return [(a, b, i if 0 <= i < n else -1) for a, b, i in zip(off, off[1:], ids)]


def lora_forward64(c, dt, segs, with_base=True):
    """out, V and their bounds."""
    X, A, B, s = (c[k].to(D) for k in ("X", "A", "B", "scaling"))
    T, K = X.shape
    N, R = B.shape[1], B.shape[2]
    half = 0.0 if dt == "f32" else 2.0 ** -17
    y = c["base"].to(D).clone() if with_base else torch.zeros((T, N), dtype=D)
    V, eV = torch.zeros((T, R), dtype=D), torch.zeros((T, R), dtype=D)
    e = torch.zeros_like(y)
    mag = y.abs()
    for lo, hi, a in segs:
        if a < 0 or hi <= lo:
            continue
        V[lo:hi] = X[lo:hi] @ A[a].t()
        eV[lo:hi] = 1.01 * K * U * (X[lo:hi].abs() @ A[a].abs().t())
        va = V[lo:hi].abs() + eV[lo:hi]
        d = s[a] * (va @ B[a].abs().t())
        y[lo:hi] += s[a] * (V[lo:hi] @ B[a].t())
        e[lo:hi] = s[a] * (eV[lo:hi] @ B[a].abs().t()) + d * (half + 1.01 * (2 * R + 4) * U)
        mag[lo:hi] += d
    e += 2 * U * mag
    return y, e + (y.abs() + e) * half_step(dt) + TINY[dt], V, eV


def lora_backward64(c, dt, segs, with_base=True):
    """grad_X, grad_A, grad_B and their bounds, with the forward's V in 64 bits."""
    X, A, B, s, G = (c[k].to(D) for k in ("X", "A", "B", "scaling", "G"))
    T, K = X.shape
    n, N, R = B.shape
    half = 0.0 if dt == "f32" else 2.0 ** -17
    gX = c["base_grad"].to(D).clone() if with_base else torch.zeros((T, K), dtype=D)
    eX, mag = torch.zeros_like(gX), gX.abs()
    gA, eA, gB, eB = torch.zeros_like(A), torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(B)
    for a in range(n):
        rows = torch.tensor([t for lo, hi, i in segs if i == a for t in range(lo, hi)], dtype=torch.long)
        if rows.numel() == 0:
            continue
        x, g, m = X[rows], G[rows], rows.numel()
        V = x @ A[a].t()
        eV = 1.01 * K * U * (x.abs() @ A[a].abs().t())
        dV = s[a] * (g @ B[a])
        edV = 1.01 * (N + 2) * U * s[a] * (g.abs() @ B[a].abs())
        va, da = V.abs() + eV, dV.abs() + edV
        gX[rows] += dV @ A[a]
        eX[rows] += edV @ A[a].abs() + (half + 1.01 * (2 * R + 4) * U) * (da @ A[a].abs())
        mag[rows] += da @ A[a].abs()
        # half: the split; 2 m: the products of both parts in one sum
        gA[a] = dV.t() @ x
        eA[a] = edV.t() @ x.abs() + (half + 1.01 * (2 * m + 4) * U) * (da.t() @ x.abs())
        gB[a] = s[a] * (g.t() @ V)
        eB[a] = s[a] * (g.abs().t() @ eV + (half + 1.01 * (2 * m + 4) * U) * (g.abs().t() @ va))
    eX += 2 * U * mag
    h, tiny = half_step(dt), TINY[dt]
    return [(v, e + (v.abs() + e) * h + tiny) for v, e in ((gX, eX), (gA, eA), (gB, eB))]


# ---- layer norm


def norm64(X, w, b, eps, dt):
    """out, mean, rstd and their bounds. The variance is a sum of squares of differences to the fp32 mean, whose own
    error e moves it by e^2 only."""
    X, w = X.to(D), w.to(D)
    C = X.shape[1]
    mean = X.mean(1, keepdim=True)
    em = 1.01 * (C + 2) * U * X.abs().mean(1, keepdim=True)
    var = ((X - mean) ** 2).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    # each difference: one rounding of (x - mean) and the mean's error
    ed = em + U * (X - mean).abs()
    evar = 1.01 * (C + 3) * U * var + 2 * ((X - mean).abs() * U * (X - mean).abs()).mean(1, keepdim=True) + em ** 2 \
        + 2 * em * (X - mean).mean(1, keepdim=True).abs()
    er = rstd * (0.51 * (evar + U * (var + eps)) / (var + eps) + 4 * U)
    h = (X - mean) * rstd
    eh = ed * rstd + (X - mean).abs() * er + ed * er + U * h.abs()
    bb = b.to(D) if b is not None else torch.zeros_like(w)
    y = h * w + bb
    ey = eh * w.abs() + 2 * U * ((h * w).abs() + bb.abs())
    return (y, ey + (y.abs() + ey) * half_step(dt) + TINY[dt]), (mean[:, 0], em[:, 0]), (rstd[:, 0], er[:, 0])


def norm_backward64(G, X, mean, rstd, w, dt, wdt):
    """grad_X, grad_weight, grad_bias and bounds, from the fp32 mean and rstd that the call is given."""
    G, X, w = G.to(D), X.to(D), w.to(D)
    T, C = X.shape
    mean, rstd = mean.to(D)[:, None], rstd.to(D)[:, None]
    h = (X - mean) * rstd
    eh = 2.02 * U * h.abs()
    u = G * w
    eu = U * u.abs()
    m1, m2 = u.mean(1, keepdim=True), (u * h).mean(1, keepdim=True)
    e1 = 1.01 * (C + 3) * U * u.abs().mean(1, keepdim=True)
    e2 = 1.01 * (C + 6) * U * (u * h).abs().mean(1, keepdim=True)
    gx = rstd * (u - m1 - h * m2)
    ex = rstd * (eu + e1 + h.abs() * e2 + eh * m2.abs() + 5 * U * (u.abs() + m1.abs() + (h * m2).abs()))
    gw, gb = (G * h).sum(0), G.sum(0)
    ew = 1.01 * (T + 4) * U * (G * h).abs().sum(0)
    eb = 1.01 * (T + 1) * U * G.abs().sum(0)
    hd, hw = half_step(dt), half_step(wdt)
    return [(gx, ex + (gx.abs() + ex) * hd + TINY[dt]), (gw, ew + (gw.abs() + ew) * hw + TINY[wdt]),
            (gb, eb + (gb.abs() + eb) * hw + TINY[wdt])]


# ---- AdamW


BLOCK = 256


def e4m3(y):
    """Nearest e4m3 value of |y| <= 448, ties to even, by arithmetic in 64 bits."""
    mag = y.abs()
    step = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(y) * torch.round(mag / step) * step


def pack64(x, positive):
    """(codes as values, scales, step of each value) of a 1-D float64 tensor in blocks of 256 from its start."""
    n = x.numel()
    pad = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=D)
    pad[:n] = x
    b = pad.view(-1, BLOCK)
    top = b.abs().amax(1)
    scale = torch.full_like(top, 2.0 ** -126)
    for i, t in enumerate(top.tolist()):
        while t / scale[i] > 448.0:
            scale[i] *= 2
    y = b / scale[:, None]
    if positive:
        y = torch.where(b > 0, y.clamp(min=2.0 ** -9), y)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return e4m3(y).view(-1)[:n], scale, step.view(-1)[:n]


def adamw64(w, g, m, v, step, lr, b1, b2, eps, wd, c=1.0):
    g = g * c
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    w = w * (1 - lr * wd) - lr / (1 - b1 ** step) * m / (torch.sqrt(v) / (1 - b2 ** step) ** 0.5 + eps)
    return w, m, v
