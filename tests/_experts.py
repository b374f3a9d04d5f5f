"""Plain 64-bit forms of the experts' operators and the gradient norm, on the CPU or the GPU, and the bounds that the
kernels' results are held to."""
import math

import torch

from tests._gpu import TORCH

HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}        # half a step, relative to the value
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}                     # half a step below the smallest normal value
d = torch.float64


def rounded(y, slack, dt):
    """Bound on |D(y') - y| where |y' - y| <= slack: the slack, and one rounding of a value up to |y| + slack."""
    return slack + HALF[dt] * (y.abs() + slack) + TINY[dt]


def check(got, y, bound, what):
    assert got.shape == y.shape, (what, got.shape, y.shape)
    err = (got.to(d) - y).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: {float(got[i])} "
                             f"against {float(y[i])}, bound {float(bound[i])}")


# ---- routing --------------------------------------------------------------------------------------------------------


def sort(ids, E):
    """Counting sort in Python integers."""
    T, k = ids.shape
    flat = ids.reshape(-1).tolist()
    off, token, position = [0], [], [-1] * (T * k)
    for e in range(E):
        for i, x in enumerate(flat):
            if x == e:
                position[i] = len(token)
                token.append(i // k)
        off.append(len(token))
    token += [-1] * (T * k - len(token))
    i32 = torch.int32
    return torch.tensor(off, dtype=i32), torch.tensor(token, dtype=i32), torch.tensor(position, dtype=i32).view(T, k)


def choices(T, k, E, seed, drop=0.0, skew=0.7):
    g = torch.Generator().manual_seed(seed)
    if E == 0:
        return torch.full((T, k), -1)
    score = torch.randn((T, E), generator=g) + skew * torch.randn(E, generator=g)
    ids = score.topk(min(k, E), 1).indices
    if k > E:
        ids = ids.repeat(1, -(-k // E))[:, :k]
    ids[torch.rand((T, k), generator=g) < drop] = -1
    return ids


# ---- products -------------------------------------------------------------------------------------------------------


def weights(E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn((E, N, K), generator=g) * max(K, 1) ** -0.5
    s = w.half().float().abs().amax(2) if K else torch.zeros((E, N))
    CB = torch.where(s[..., None] > 0, torch.round(w.half().float() * (127.0 / s)[..., None]), 0.0)
    return CB.clamp(-127, 127).to(torch.int8), s


def inputs(T, K, dt, seed, outliers=2):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g)
    if K and outliers:
        x[:, torch.randperm(K, generator=g)[:outliers]] *= 20
    return x.to(TORCH[dt])


def quantized(X, tau):
    """codes, scales, outlier part: as the quantizer defines them, in 64 bits with its two fp32 roundings."""
    x = X.to(torch.float16).to(d)
    on = tau > 0 and tau < math.inf
    cols = (x.abs() > tau).any(0) if on and x.shape[0] else torch.zeros(x.shape[1], dtype=torch.bool, device=x.device)
    inner = torch.where(cols, 0.0, x)
    top = inner.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0], dtype=d, device=x.device)
    inv = (torch.full_like(top, 127.0) / torch.where(top > 0, top, 1.0)).float().to(d)
    codes = torch.where((top > 0)[:, None], torch.round((inner * inv[:, None]).float().to(d)), 0.0)
    return codes, top, torch.where(cols, x, 0.0), int(cols.sum())


def dequantized(cb, scb):
    unit = (scb.to(d) * torch.tensor(1 / 127, dtype=torch.float32).to(d).item()).float().to(d)
    return (cb.to(d) * unit[:, None]).float().to(torch.float16).to(d)


def row_experts(off, ids, R, E):
    """The expert of each row, -1 for none."""
    off = off.tolist()
    who = [-1] * R
    for j in range(len(off) - 1):
        e = j if ids is None else int(ids[j])
        for r in range(0 if j == 0 else off[j], off[j + 1]):
            who[r] = e if 0 <= e < E else -1
    return who


def forward(X, CB, SCB, off, ids=None, rows=None, tau=6.0):
    """(y, slack) of the products in 64 bits. slack: the int32 sum's conversion, the scales' three products and the last
    one round once each; every outlier column adds one rounded (or truncated) sum of fp32."""
    T = X.shape[0]
    E, N, _ = CB.shape
    codes, top, out, n_out = quantized(X, tau)
    R = T if rows is None else rows.numel()
    y = torch.zeros((R, N), dtype=d, device=X.device)
    slack = torch.zeros_like(y)
    who = row_experts(off, ids, R, E)
    for e in sorted(set(who) - {-1}):
        w, dq = CB[e].to(d), dequantized(CB[e], SCB[e])
        r = torch.tensor([i for i, x in enumerate(who) if x == e], device=X.device)
        t = r if rows is None else rows.to(X.device)[r].long()
        ok = (t >= 0) & (t < T)
        r, t = r[ok], t[ok]
        whole = (codes[t] @ w.t()) * top[t][:, None] * (SCB[e].to(d) / 127 ** 2)
        parts = out[t].abs() @ dq.abs().t()
        y[r] = whole + out[t] @ dq.t()
        slack[r] = 6 * 2.0 ** -24 * whole.abs() + (n_out + 4) * 2.0 ** -23 * (whole.abs() + parts) * (n_out > 0)
    return y, slack


def backward(G, CB, SCB, off, ids=None):
    """(gX, slack): fp16 products are exact in fp32; a matrix instruction adds 16 of them, N / 16 instructions follow
    each other, so the bound counts N / 16 + 16 truncated sums of the magnitudes."""
    R, N = G.shape
    E, _, K = CB.shape
    g = G.to(torch.float16).to(d)
    y = torch.zeros((R, K), dtype=d, device=G.device)
    slack = torch.zeros_like(y)
    who = row_experts(off, ids, R, E)
    for e in sorted(set(who) - {-1}):
        r = torch.tensor([i for i, x in enumerate(who) if x == e], device=G.device)
        dq = dequantized(CB[e], SCB[e])
        y[r] = g[r] @ dq
        slack[r] = (N / 16 + 16) * 2.0 ** -23 * (g[r].abs() @ dq.abs())
    return y, slack


# ---- weighted sum ---------------------------------------------------------------------------------------------------


def combine(Y, position, gate=None, base=None):
    T, k = position.shape
    N = Y.shape[1]
    y = torch.zeros((T, N), dtype=d, device=Y.device) if base is None else base.to(d)
    mag = y.abs()
    has = (position >= 0) & (position < Y.shape[0])
    for j in range(k):
        t = has[:, j].nonzero()[:, 0]
        w = 1.0 if gate is None else gate[t, j].to(d)[:, None]
        part = w * Y[position[t, j].long()].to(d)
        y = y.index_add(0, t, part)
        mag = mag.index_add(0, t, part.abs())
    return y, (k + 1) * 2.0 ** -24 * mag


def combine_backward(G, position, gate, Y, R):
    """(grad_Y with zeros where no position names a row, grad_gate, its slack)."""
    T, k = position.shape
    N = G.shape[1]
    gY = torch.zeros((R, N), dtype=d, device=G.device)
    gg = torch.zeros((T, k), dtype=d, device=G.device)
    mag = torch.zeros_like(gg)
    has = (position >= 0) & (position < R)
    for j in range(k):
        t = has[:, j].nonzero()[:, 0]
        r = position[t, j].long()
        gY[r] = G[t].to(d) * (1.0 if gate is None else gate[t, j].to(d)[:, None])
        if Y is not None:
            p = G[t].to(d) * Y[r].to(d)
            gg[t, j], mag[t, j] = p.sum(1), p.abs().sum(1)
    return gY, gg, (N / 64 + 16) * 2.0 ** -24 * mag


def combine_gradient(G, position, gate, R):
    """(grad_Y, slack) for positions of any kind: each row gets the sum over all that name it, none 0. One rounding a
    term, of the product or of the sum so far."""
    T, k = position.shape
    gY = torch.zeros((R, G.shape[1]), dtype=d, device=G.device)
    mag = torch.zeros_like(gY)
    named = torch.zeros(R, dtype=d, device=G.device)
    has = (position >= 0) & (position < R)
    for j in range(k):
        t = has[:, j].nonzero()[:, 0]
        r = position[t, j].long()
        part = G[t].to(d) * (1.0 if gate is None else gate[t, j].to(d)[:, None])
        gY, mag = gY.index_add(0, r, part), mag.index_add(0, r, part.abs())
        named = named.index_add(0, r, torch.ones_like(r, dtype=d))
    return gY, named[:, None] * 2.0 ** -24 * mag


# ---- gradient norm --------------------------------------------------------------------------------------------------


def grad_norm(grads, max_norm=math.inf, norm_type=2, c=1.0):
    """(norm, factor) in Python floats."""
    flat = [g.to(d).reshape(-1) for g in grads if g.numel()]
    if norm_type == 2:
        total = math.sqrt(math.fsum(float((g * g).sum()) for g in flat))
    else:
        total = max([0.0] + [float(g.abs().max()) for g in flat])
    norm = abs(c) * total
    return norm, c * min(1.0, max_norm / (norm + 1e-6))
