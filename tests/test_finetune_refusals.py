"""The adapters, layer norm and AdamW entry points refuse bad arguments on the
host, before any HIP call (nothing here touches a GPU), and the plain 64-bit
forms the GPU tests use are checked against differences and torch."""
import ctypes

import pytest
import torch

from tests import _finetune as F
from tests.test_abi import FAKE, L  # noqa: F401  (fixture: builds the library if it is missing)


def test_lora_forward_host_errors(L):  # noqa: F811
    f, need = L.lib.int8_lora_forward, L.lib.int8_lora_forward_workspace_bytes
    # a size that takes a workspace (small ones run without)
    base = dict(X=FAKE, dt=2, T=8, K=64000, A=FAKE, B=FAKE, s=FAKE, n=2, R=16, N=32, off=FAKE, ids=FAKE, S=3,
                base=None, out=FAKE, V=None, ws=FAKE, wsb=1 << 40, st=None)

    def call(**kw):
        a = dict(base, **kw)
        return f(*(a[k] for k in base))

    assert call(dt=3) == L.I8L_EDTYPE and call(dt=-1) == L.I8L_EDTYPE
    for k in ("T", "K", "N", "R", "n", "S"):
        assert call(**{k: -1}) == L.I8L_EINVAL, k
    for k in ("X", "A", "B", "s", "off", "out"):
        assert call(**{k: 0}) == L.I8L_EINVAL, k
    assert call(R=L.I8L_LORA_MAX_RANK + 1) == L.I8L_ESHAPE
    assert call(K=L.I8L_MAX_COLS + 1) == L.I8L_ESHAPE and call(N=L.I8L_MAX_COLS + 1) == L.I8L_ESHAPE
    assert call(T=1 << 31) == L.I8L_ESHAPE and call(S=1 << 31) == L.I8L_ESHAPE and call(n=65536) == L.I8L_ESHAPE
    assert call(T=1 << 29, S=(1 << 29) + 1) == L.I8L_ESHAPE
    assert call(T=(1 << 24) + 1) == L.I8L_ESHAPE and call(S=(1 << 20) + 1) == L.I8L_ESHAPE
    assert call(n=65535, K=16384, R=1) == L.I8L_ESHAPE       # 65535 x 16384 x 16 (the padded rank) > 2^33
    wsb = need(8, 64000, 32, 16, 3)
    assert wsb % 256 == 0 and wsb > 0
    assert call(wsb=wsb - 1) == L.I8L_EWORKSPACE and call(ws=0) == L.I8L_EWORKSPACE
    assert call(ws=FAKE + 16) == L.I8L_EINVAL
    assert call(T=0, X=0, out=0, off=0, ws=0, wsb=0) == L.I8L_OK
    assert need(-1, 64, 32, 16, 3) == 0 and need(8, 64, 32, 129, 3) == 0 and need(8, 64, 32, 16, 3) == 0


def test_lora_backward_host_errors(L):  # noqa: F811
    f, need = L.lib.int8_lora_backward, L.lib.int8_lora_backward_workspace_bytes
    base = dict(G=FAKE, X=FAKE, V=FAKE, dt=1, T=8, K=64, A=FAKE, B=FAKE, s=FAKE, n=2, R=16, N=32, off=FAKE, ids=FAKE,
                S=3, bg=None, gX=FAKE, gA=FAKE, gB=FAKE, ws=FAKE, wsb=1 << 40, st=None)

    def call(**kw):
        a = dict(base, **kw)
        return f(*(a[k] for k in base))

    assert call(dt=9) == L.I8L_EDTYPE
    for k in ("T", "K", "N", "R", "n", "S"):
        assert call(**{k: -1}) == L.I8L_EINVAL, k
    for k in ("G", "X", "V", "A", "B", "s", "off"):
        assert call(**{k: 0}) == L.I8L_EINVAL, k
    assert call(R=129) == L.I8L_ESHAPE and call(T=1 << 31) == L.I8L_ESHAPE
    wsb = need(8, 64, 32, 16, 2, 3)
    assert wsb % 256 == 0 and wsb > 0
    assert call(wsb=wsb - 1) == L.I8L_EWORKSPACE and call(ws=0) == L.I8L_EWORKSPACE
    assert call(ws=FAKE + 8) == L.I8L_EINVAL
    assert need(8, 64, 32, 16, -1, 3) == 0


def test_layer_norm_host_errors(L):  # noqa: F811
    f = L.lib.int8_layer_norm_forward
    base = dict(X=FAKE, dt=2, T=4, C=8, w=FAKE, b=None, wdt=0, eps=1e-5, out=FAKE, mean=None, rstd=None, st=None)

    def call(**kw):
        a = dict(base, **kw)
        return f(*(a[k] for k in base))

    assert call(dt=5) == L.I8L_EDTYPE and call(wdt=1) == L.I8L_EDTYPE and call(dt=0, wdt=2) == L.I8L_EDTYPE
    assert call(T=-1) == L.I8L_EINVAL and call(C=-1) == L.I8L_EINVAL
    assert call(C=L.I8L_MAX_COLS + 1) == L.I8L_ESHAPE and call(T=1 << 31) == L.I8L_ESHAPE
    for k in ("X", "w", "out"):
        assert call(**{k: 0}) == L.I8L_EINVAL, k
    assert call(eps=-1.0) == L.I8L_EINVAL and call(eps=float("nan")) == L.I8L_EINVAL
    assert call(T=0, X=0, out=0) == L.I8L_OK and call(C=0, X=0, out=0, w=0) == L.I8L_OK

    g, need = L.lib.int8_layer_norm_backward, L.lib.int8_layer_norm_backward_workspace_bytes
    bbase = dict(G=FAKE, X=FAKE, dt=2, T=4, C=8, mean=FAKE, rstd=FAKE, w=FAKE, wdt=2, gX=2 * FAKE, gw=FAKE, gb=FAKE,
                 ws=FAKE, wsb=1 << 40, st=None)

    def bcall(**kw):
        a = dict(bbase, **kw)
        return g(*(a[k] for k in bbase))

    assert bcall(dt=4) == L.I8L_EDTYPE and bcall(wdt=1) == L.I8L_EDTYPE
    for k in ("G", "X", "mean", "rstd", "w"):
        assert bcall(**{k: 0}) == L.I8L_EINVAL, k
    assert bcall(gX=FAKE) == L.I8L_EINVAL                     # grad_X over G while the weight's gradient reads G
    assert bcall(C=0, G=0, X=0) == L.I8L_OK
    if need(4, 8):
        assert bcall(wsb=need(4, 8) - 1) == L.I8L_EWORKSPACE
    assert bcall(ws=FAKE + 8) == L.I8L_EINVAL
    assert need(-1, 8) == 0 and need(4, L.I8L_MAX_COLS + 1) == 0


def test_adamw_host_errors(L):  # noqa: F811
    T = L.AdamWTensor
    fill, size = L.lib.int8_adamw_table_fill, L.lib.int8_adamw_table_bytes

    def one(**kw):
        a = dict(p=FAKE, g=FAKE, m=FAKE, v=FAKE, m_scale=FAKE, v_scale=FAKE, master=None, n=5000, dtype=2,
                 state_bits=8)
        a.update(kw)
        return (T * 1)(T(*a.values()))

    def call(t, count=1, short=0, chunks=True):
        n = size(t, count)
        buf = (ctypes.c_uint8 * max(n, 1))()
        c = ctypes.c_int64(-1)
        return fill(t, count, ctypes.addressof(buf), n - short, ctypes.byref(c) if chunks else None), c.value

    rc, chunks = call(one())
    assert rc == L.I8L_OK and chunks >= 1
    assert call(one(dtype=3))[0] == L.I8L_EDTYPE
    assert call(one(state_bits=16))[0] == L.I8L_EINVAL
    for k in ("p", "g", "m", "v", "m_scale", "v_scale"):
        assert call(one(**{k: None}))[0] == L.I8L_EINVAL, k
    assert call(one(m_scale=None, v_scale=None, state_bits=32))[0] == L.I8L_OK
    assert call(one(), short=1)[0] == L.I8L_EWORKSPACE
    assert call(one(), chunks=False)[0] == L.I8L_EINVAL
    assert size(one(n=-1), 1) == 0 and size(one(n=1 << 41), 1) == 0 and size(one(), -1) == 0
    assert call(one(n=0, p=None, g=None, m=None, v=None, m_scale=None, v_scale=None)) == (L.I8L_OK, 0)

    f = L.lib.int8_adamw_step
    base = dict(table=FAKE, count=1, chunks=3, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, step=1, gs=None, fi=None,
                st=None)

    def step(**kw):
        a = dict(base, **kw)
        return f(*(a[k] for k in base))

    nan, inf = float("nan"), float("inf")
    for kw in (dict(step=0), dict(b1=1.0), dict(b1=-0.1), dict(b2=nan), dict(lr=-1.0), dict(lr=inf), dict(eps=nan),
               dict(wd=-0.1), dict(wd=inf), dict(table=0), dict(table=FAKE + 4), dict(chunks=-1), dict(count=-1)):
        assert step(**kw) == L.I8L_EINVAL, kw
    assert step(chunks=0, table=0) == L.I8L_OK


def test_binding_refusals(L):  # noqa: F811
    import int8_quantized_linear_rowwise_amd as I8
    h = torch.float16
    X, A, B, s = torch.zeros(4, 16, dtype=h), torch.zeros(2, 8, 16, dtype=h), torch.zeros(2, 6, 8, dtype=h), torch.ones(2)
    G, V = torch.zeros(4, 6, dtype=h), torch.zeros(4, 8)
    off = torch.tensor([0, 4], dtype=torch.int32)
    w = torch.ones(16, dtype=h)
    mean = torch.zeros(4)
    bad = [
        lambda: I8.lora_forward(X, A, B, s),                                     # not on a GPU
        lambda: I8.lora_forward(X[0], A, B, s),
        lambda: I8.lora_forward(X, A[:, :, :8], B, s),
        lambda: I8.lora_forward(X, A, B[:, :, :4], s),
        lambda: I8.lora_forward(X, A.float(), B, s),
        lambda: I8.lora_forward(X, A, B, s.double()),
        lambda: I8.lora_forward(X, A, B, s[:1]),
        lambda: I8.lora_forward(X, A, B, s, off.long()),
        lambda: I8.lora_forward(X, A, B, s, off, torch.zeros(2, dtype=torch.int32)),
        lambda: I8.lora_forward(X, A, B, s, off, torch.zeros(1)),
        lambda: I8.lora_forward(X, A, B, s, base=G[:3]),
        lambda: I8.lora_forward(X, A, B, s, out=G.float()),
        lambda: I8.lora_forward(X, A, B, s, v=V.half()),
        lambda: I8.lora_forward(X, A, B, s, workspace=torch.zeros(1, dtype=torch.uint8)),
        lambda: I8.lora_backward(G, X, V.half(), A, B, s),
        lambda: I8.lora_backward(G[:3], X, V, A, B, s),
        lambda: I8.lora_backward(G.float(), X, V, A, B, s),
        lambda: I8.lora_backward(G, X, V, A, B, s, grad_A=A[:1]),
        lambda: I8.lora_backward(G, X, V, A, B, s),
        lambda: I8.layer_norm_forward(X, w),
        lambda: I8.layer_norm_forward(X, w[:8]),
        lambda: I8.layer_norm_forward(X, w.bfloat16()),
        lambda: I8.layer_norm_forward(X, w, w.float()),
        lambda: I8.layer_norm_forward(X, w, out=X.float()),
        lambda: I8.layer_norm_backward(X, X[:2], mean, mean, w),
        lambda: I8.layer_norm_backward(X, X, mean[:2], mean, w),
        lambda: I8.layer_norm_backward(X, X, mean.half(), mean, w),
        lambda: I8.layer_norm_backward(X, X, mean, mean, w, grad_weight=w.float()),
        lambda: I8.AdamWPlan([], [], [], []),
        lambda: I8.AdamWPlan([w], [], [w.float()], [w.float()]),
        lambda: I8.AdamWPlan([w], [w.float()], [w.float()], [w.float()]),
        lambda: I8.AdamWPlan([w], [w], [w], [w]),
        lambda: I8.AdamWPlan([w], [w], [w.float()], [w.to(torch.float8_e4m3fn)]),
        lambda: I8.AdamWPlan([w], [w], [w.to(torch.float8_e4m3fn)], [w.to(torch.float8_e4m3fn)]),
        lambda: I8.AdamWPlan([w], [w], [w.float()], [w.float()], master=[w]),
        lambda: I8.AdamWPlan([w], [w], [w.float()], [w.float()]),
        lambda: I8.adamw_state(w, bits=4),
        lambda: I8.AdamW([torch.nn.Parameter(w)], state_bits=16),
        lambda: I8.Int8LoraLinear(torch.zeros(8, 16), rank=129),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)
    with pytest.raises(TypeError):
        I8.AdamWPlan([w.double()], [w.double()], [w.float()], [w.float()])
    st = I8.adamw_state(torch.zeros(300, dtype=h), bits=8, master=True)
    assert st["m"].dtype == torch.float8_e4m3fn and st["m_scale"].shape == (2,) and st["master"].dtype == torch.float32


def test_plain_lora_gradients_against_differences():
    """The plain 64-bit gradients equal central differences of the plain forward."""
    c = {k: v.double() for k, v in F.lora_inputs("f32", 7, 5, 4, 3, 2, 1).items()}
    segs = F.segments_of([0, 3, 3, 5, 7], [1, 0, -1, 1], 2, 7)

    def loss(c):
        return float((F.lora_forward64(c, "f32", segs)[0] * c["G"]).sum())

    grads = dict(zip("XAB", (g for g, _ in F.lora_backward64(c, "f32", segs, with_base=False))))
    for name, g in grads.items():
        for i in range(g.numel()):
            d = dict(c)
            h = 1e-4
            d[name] = c[name].clone()
            d[name].view(-1)[i] += h
            up = loss(d)
            d[name] = c[name].clone()
            d[name].view(-1)[i] -= h
            # the loss is a product of at most three factors: differences are exact up to h^2 and rounding
            assert abs((up - loss(d)) / (2 * h) - float(g.view(-1)[i])) < 1e-6, (name, i)


def test_plain_norm_and_adamw_against_torch():
    X, w, b, G = (F.randn(s, "f32", i).double() for i, s in enumerate(((6, 40), (40,), (40,), (6, 40))))
    Xr, wr, br = (t.clone().requires_grad_(True) for t in (X, w, b))
    y = torch.nn.functional.layer_norm(Xr, (40,), wr, br, 1e-5)
    (y * G).sum().backward()
    (yy, _), (mean, _), (rstd, _) = F.norm64(X, w, b, 1e-5, "f32")
    assert torch.allclose(y.detach(), yy, rtol=1e-12, atol=1e-12)
    got = F.norm_backward64(G, X, mean, rstd, w, "f32", "f32")
    for (g, _), t in zip(got, (Xr, wr, br)):
        assert torch.allclose(g, t.grad, rtol=1e-10, atol=1e-12)
    p = torch.nn.Parameter(F.randn((50,), "f32", 9).double())
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().clone(), torch.zeros(50, dtype=F.D), torch.zeros(50, dtype=F.D)
    for k in range(1, 5):
        p.grad = F.randn((50,), "f32", 20 + k).double()
        opt.step()
        q, m, v = F.adamw64(q, p.grad, m, v, k, 1e-2, 0.8, 0.95, 1e-6, 0.1)
        assert torch.allclose(p.detach(), q, rtol=1e-12, atol=1e-14)


def test_plain_codes_against_torch():
    """The 64-bit e4m3 rounding equals torch's conversion for every fp32 value tried, and blocks use the least scale."""
    x = torch.cat([torch.linspace(-448, 448, 5001), torch.randn(5000) * 0.01, torch.tensor([0.0, 2.0 ** -10,
                                                                                           3 * 2.0 ** -10, 448.0])])
    assert torch.equal(F.e4m3(x.double()), x.to(torch.float8_e4m3fn).double())
    code, scale, _ = F.pack64(torch.tensor([448.0, 1.0, 0.0] + [0.0] * 253 + [449.0] + [1e-9] * 40).double(), True)
    assert scale.tolist() == [1.0, 2.0]
    assert code[0] == 448 and code[256] == 224 and code[257] == 2.0 ** -9 and code[2] == 0
