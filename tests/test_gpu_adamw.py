"""GPU parity of the AdamW step over many tensors, states in 32 and in 8 bits,
against the plain 64-bit forms, and of the optimizer built on it."""
import weakref

import numpy as np
import pytest
import torch

from tests import _finetune as F

pytestmark = pytest.mark.gpu
U, D = F.U, F.D
H = dict(lr=3e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.05)
SIZES = [1, 31, 255, 256, 257, 2048, 2049, 5000, 4096 * 16, 0, 7]


@pytest.fixture(scope="module")
def I8():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import int8_quantized_linear_rowwise_amd as I8
    return I8


def make(dt, n, bits, master, seed, offset=0):
    """One tensor's p, g and state on the GPU; `offset` shifts each inside its storage."""
    def put(x):
        s = torch.zeros(x.numel() + offset, dtype=x.dtype)
        s.view(torch.uint8)[:] = 0
        s[offset:] = x
        return s.cuda()[offset:]

    w, g = F.randn((n,), "f32", seed, 0.5), F.randn((n,), dt, seed + 1, 0.01)
    m, q = F.randn((n,), "f32", seed + 2, 0.01), F.randn((n,), "f32", seed + 3).exp() * 0.01
    s = dict(p=put(w.to(F.DT[dt])), g=put(g), master=put(w) if master else None)
    if bits == 8:
        for k, x, pos in (("m", m, False), ("v", q, True)):
            code, scale, _ = F.pack64(x.double(), pos)
            raw = code.float().to(torch.float8_e4m3fn).view(torch.uint8)
            s[k], s[k + "_scale"] = put(raw).view(torch.float8_e4m3fn), put(scale.float())
    else:
        s["m"], s["v"] = put(m), put(q * q)
    return s


def plan(I8, ts, bits, master):
    get = lambda k: [t[k] for t in ts]  # noqa: E731
    low = bits == 8
    return I8.AdamWPlan(get("p"), get("g"), get("m"), get("v"), get("m_scale") if low else None,
                        get("v_scale") if low else None, get("master") if master else None)


def unpack(code, scale):
    n = code.numel()
    return code.cpu().float().to(D) * scale.cpu().to(D).repeat_interleave(F.BLOCK)[:n]


def before(t, bits):
    """State of a tensor in 64 bits: w, g, m, v."""
    w = (t["master"] if t["master"] is not None else t["p"]).cpu().to(D)
    if bits == 8:
        return w, t["g"].cpu().to(D), unpack(t["m"], t["m_scale"]), unpack(t["v"], t["v_scale"]) ** 2
    return w, t["g"].cpu().to(D), t["m"].cpu().to(D), t["v"].cpu().to(D)


def check_after(t, was, bits, dt, step, what, c=1.0, h=H):
    w, g, m, v = was
    w1, m1, v1 = F.adamw64(w, g, m, v, step, h["lr"], h["b1"], h["b2"], h["eps"], h["wd"], c)
    gc = (g * c).abs()
    # m: g c, two products, one sum; the factors themselves are rounded to fp32. v: its square too
    em = 5 * U * ((h["b1"] * m).abs() + (1 - h["b1"]) * gc)
    ev = 8 * U * v1
    q1, eq = torch.sqrt(v1), 5 * U * torch.sqrt(v1)
    upd = (w1 - w * (1 - h["lr"] * h["wd"])).abs()
    rel = em / m1.abs().clamp(min=1e-300)
    ew = 3 * U * w.abs() + upd * (rel + 14 * U) + U * w1.abs()
    F.assert_within(t["p"], w1, ew + (w1.abs() + ew) * (F.half_step(dt) if dt != "f32" else 0) + F.TINY[dt], what + " p")
    if t["master"] is not None:
        F.assert_within(t["master"], w1, ew, what + " master")
        assert torch.equal(t["p"].cpu(), t["master"].cpu().to(t["p"].dtype)), what
    if bits == 32:
        F.assert_within(t["m"], m1, em, what + " m")
        F.assert_within(t["v"], v1, ev, what + " v")
        return
    for name, x, e, pos in (("m", m1, em, False), ("v", q1, eq, True)):
        if x.numel() == 0:
            continue
        scale = t[name + "_scale"].cpu().to(D)
        # the scale is a power of two, and the least that fits a block maximum within its error
        assert torch.equal(torch.exp2(torch.log2(scale).round()), scale), what
        pad = torch.zeros(scale.numel() * F.BLOCK, dtype=D)
        pad[:x.numel()] = x.abs()
        top, etop = pad.view(-1, F.BLOCK).amax(1), 1e-6
        small = scale == 2.0 ** -126
        assert (top * (1 - etop) <= 448 * scale).all() and ((top * (1 + etop) > 224 * scale) | small).all(), what
        unit = scale.repeat_interleave(F.BLOCK)[:x.numel()]
        y = x / unit
        if pos:
            y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
        step_y = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        # half a step of e4m3 (a full binade's at its upper end), and the value's own error
        F.assert_within(t[name].cpu().float().to(D), y, step_y / 2 * 1.0001 + e / unit, f"{what} {name} codes")
        assert not pos or (t[name].cpu().float()[x > 0] > 0).all(), what


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dt,master", [("f32", False), ("bf16", False), ("bf16", True), ("f16", False), ("f16", True)])
@pytest.mark.parametrize("offset", [0, 1])
def test_sizes(I8, dt, master, bits, offset):
    print(f"\n  [{dt} master={master} bits={bits} offset={offset}]", flush=True)
    ts = [make(dt, n, bits, master, 10 * i, offset) for i, n in enumerate(SIZES)]
    pl = plan(I8, ts, bits, master)
    for step in (1, 2, 50):
        was = [before(t, bits) for t in ts]
        pl.step(step, H["lr"], (H["b1"], H["b2"]), H["eps"], H["wd"])
        torch.cuda.synchronize()
        for n, t, b in zip(SIZES, ts, was):
            check_after(t, b, bits, dt, step, f"n={n} step={step}")


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_types_in_one_plan(I8, bits):
    kinds = [("f32", 300), ("bf16", 5000), ("f16", 77), ("f32", 4096), ("bf16", 256)]
    ts = [make(dt, n, bits, False, 7 * i) for i, (dt, n) in enumerate(kinds)]
    pl = plan(I8, ts, bits, False)
    was = [before(t, bits) for t in ts]
    pl.step(3, H["lr"], (H["b1"], H["b2"]), H["eps"], H["wd"])
    for (dt, n), t, b in zip(kinds, ts, was):
        check_after(t, b, bits, dt, 3, f"{dt} n={n}")


@pytest.mark.parametrize("bits", [32, 8])
def test_grad_scale_and_skipping(I8, bits):
    t = make("bf16", 3000, bits, True, 3)
    pl = plan(I8, [t], bits, True)
    c, inf = torch.tensor([0.25], device="cuda:0"), torch.tensor([1.0], device="cuda:0")
    copy = {k: v.clone() for k, v in t.items() if v is not None}
    pl.step(4, H["lr"], (H["b1"], H["b2"]), H["eps"], H["wd"], grad_scale=c, found_inf=inf)
    torch.cuda.synchronize()
    for k, v in copy.items():
        assert torch.equal(t[k].view(torch.uint8), v.view(torch.uint8)), k
    was = before(t, bits)
    pl.step(4, H["lr"], (H["b1"], H["b2"]), H["eps"], H["wd"], grad_scale=c, found_inf=inf * 0)
    check_after(t, was, bits, "bf16", 4, "scaled", c=0.25)
    with pytest.raises(ValueError):
        pl.step(4, 1e-3, grad_scale=c.cpu())
    with pytest.raises(ValueError):
        pl.step(4, 1e-3, found_inf=inf.double())
    with pytest.raises(I8.Int8LinError):
        pl.step(0, 1e-3)


def test_8bit_codes_equal_the_definition(I8):
    """With beta1 = beta2 = 0 the new states are the gradient and its magnitude: codes and scales have to equal the
    64-bit definition's bit for bit, from the smallest to the largest gradients and at every rounding border."""
    g = torch.Generator().manual_seed(5)
    top = torch.exp2(torch.randint(-60, 60, (64,), generator=g).float())          # one scale range a block
    x = torch.randn(64, 256, generator=g) * torch.exp2(torch.randint(-20, 1, (64, 256), generator=g).float())
    # borders: every midpoint of two codes, both signs, in two blocks whose largest value is 448
    codes = torch.arange(0, 0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (codes[:-1] + codes[1:]) / 2
    x[:2] = 0
    x[0, :125], x[0, 125], x[1, :125], x[1, 125] = mid[:125], 448, -mid[:125], -448
    top[:2] = 1
    x = (x * top[:, None]).reshape(-1)
    n = x.numel()
    dev = lambda v: v.cuda()  # noqa: E731
    t = dict(p=dev(torch.zeros(n)), g=dev(x), master=None, **I8.adamw_state(torch.zeros(n, device="cuda:0"), 8))
    plan(I8, [t], 8, False).step(1, 1e-3, (0.0, 0.0), 1e-8, 0.0)
    torch.cuda.synchronize()
    # every operation is rounded to fp32: the root of fl(g g), which is |g| unless g g leaves fp32's normal range (the
    # blocks with the smallest gradients reach its denormals)
    root = torch.from_numpy(np.sqrt(np.square(x.numpy(), dtype=np.float32), dtype=np.float32))
    assert (root != x.abs()).any() and (root == x.abs())[x.abs() > 1e-18].all()
    for k, want, pos in (("m", x.double(), False), ("v", root.double(), True)):
        code, scale, _ = F.pack64(want, pos)
        assert torch.equal(t[k + "_scale"].cpu().double(), scale), k
        assert torch.equal(t[k].cpu().float().double(), code), k


def test_8bit_special_blocks(I8):
    """Zeros stay zeros with nothing divided by nothing; an infinity or NaN marks its own block alone."""
    n = 256 * 5
    t = dict(p=torch.ones(n, device="cuda:0"), g=torch.zeros(n, device="cuda:0"), master=None,
             **I8.adamw_state(torch.zeros(n, device="cuda:0"), 8))
    t["g"][256 + 3], t["g"][512 + 5] = float("nan"), float("inf")
    t["g"][768:1024] = torch.linspace(1e-30, 1.0, 256, device="cuda:0")
    t["g"][1024] = 1e-42                                            # denormal
    plan(I8, [t], 8, False).step(1, 1e-2, (0.9, 0.99), 1e-8, 0.0)
    torch.cuda.synchronize()
    p, ms, vs = t["p"].cpu(), t["m_scale"].cpu(), t["v_scale"].cpu()
    assert (p[:256] == 1).all() and not t["m"].cpu().float()[:256].any() and not t["v"].cpu().float()[:256].any()
    assert torch.isnan(ms[1:3]).all() and torch.isnan(vs[1:3]).all() and torch.isfinite(ms[[0, 3, 4]]).all()
    assert torch.isnan(p[259]) and torch.isnan(p[517]) and (p[256:259] == 1).all() and (p[260:512] == 1).all()
    q = t["v"].cpu().float()[768:1024]
    assert (q[1:] > 0).all() and torch.isfinite(p[768:]).all() and ms[4] == 2.0 ** -126


@pytest.mark.parametrize("bits", [32, 8])
def test_same_bits_whatever_the_path(I8, bits):
    """Shifted (scalar) and aligned (wide) tensors of the same values end with the same bits, on a side stream and in
    a replayed graph too."""
    a, b = make("bf16", 5000, bits, True, 6), make("bf16", 5000, bits, True, 6, offset=1)
    pa, pb = plan(I8, [a], bits, True), plan(I8, [b], bits, True)

    def same():
        torch.cuda.synchronize()
        for k, v in a.items():
            if v is not None:
                assert torch.equal(v.contiguous().view(torch.uint8), b[k].clone().view(torch.uint8)), k

    pa.step(1, 1e-3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pb.step(1, 1e-3)
    same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.step(2, 1e-3)
    for i in range(3):
        new = F.randn((5000,), "bf16", 60 + i, 0.01).cuda()
        a["g"].copy_(new)
        b["g"].copy_(new)
        torch.cuda.synchronize()
        g.replay()
        pb.step(2, 1e-3)
        same()


def test_optimizer_matches_torch(I8):
    """32-bit states, fp32 parameters: ten steps stay within ten steps' roundings of torch's AdamW, with gradients
    that come and go, two groups and a saved and loaded state."""
    g = torch.Generator().manual_seed(8)
    shapes = [(33, 5), (4096,), (1,), (16, 64)]
    P = [torch.nn.Parameter(torch.randn(s, generator=g).cuda()) for s in shapes]
    Q = [torch.nn.Parameter(p.detach().double()) for p in P]
    mk = lambda cls, X, **kw: cls([dict(params=X[:2], lr=1e-2), dict(params=X[2:], lr=3e-3, weight_decay=0.1)],  # noqa: E731
                                  betas=(0.8, 0.9), eps=1e-6, **kw)
    ours, ref = mk(I8.AdamW, P), mk(torch.optim.AdamW, Q)
    for step in range(10):
        for i, (p, q) in enumerate(zip(P, Q)):
            p.grad = None if (i == 1 and step in (2, 3)) else torch.randn(p.shape, generator=g).cuda()
            q.grad = None if p.grad is None else p.grad.double()
        ours.step()
        ref.step()
        if step == 5:
            state = ours.state_dict()
            ours = mk(I8.AdamW, P)
            ours.load_state_dict(state)
    for p, q in zip(P, Q):
        # each step's update is at most lr * a few, off by some 20 u of itself, and w is rounded once
        lim = 10 * (2 * U * q.detach().abs().cpu() + 40 * U * 1e-2 * 3) + 2 * U
        F.assert_within(p, q.detach(), lim, "parameters")


def test_optimizer_8bit_learns_and_keeps_its_types(I8):
    """A least-squares problem: with 8-bit states and a bf16 parameter with its fp32 master the loss falls as with
    32-bit states, and a saved state comes back in its own types."""
    g = torch.Generator().manual_seed(9)
    A, target = torch.randn(512, 300, generator=g).cuda(), torch.randn(300, generator=g).cuda()
    losses = {}
    for bits in (32, 8):
        p = torch.nn.Parameter(torch.zeros(300, dtype=torch.bfloat16, device="cuda:0"))
        opt = I8.AdamW([p], lr=2e-2, weight_decay=0.0, state_bits=bits, master=True)
        for step in range(200):
            opt.zero_grad(set_to_none=step % 2 == 0)
            loss = ((A @ (p.float() - target)) ** 2).mean()
            loss.backward()
            opt.step()
            if step == 100:
                saved = opt.state_dict()
                opt = I8.AdamW([p], lr=2e-2, weight_decay=0.0, state_bits=bits, master=True)
                opt.load_state_dict(saved)
                s = opt.state[p]
                assert s["m"].dtype == (torch.float8_e4m3fn if bits == 8 else torch.float32)
                assert s["master"].dtype == torch.float32 and s["step"] == 101
        losses[bits] = float(loss.detach())
    first = float(((A @ target) ** 2).mean())
    assert losses[32] < 1e-2 * first and losses[8] < 1e-2 * first, losses


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_move_are_not_held(I8, bits):
    """Dropped gradients are freed; new ones at other addresses, in other types or layouts are seen for what they are."""
    g = torch.Generator().manual_seed(10)
    draw = lambda: torch.randn(48, 48, generator=g).cuda()  # noqa: E731
    p, q = (torch.nn.Parameter(torch.ones(48, 48, device="cuda:0")) for _ in range(2))
    ours, still = I8.AdamW([p], state_bits=bits), I8.AdamW([q], state_bits=bits)
    q.grad = torch.empty_like(q)
    for step in range(4):
        new = draw()
        p.grad = new.clone()
        q.grad.copy_(new)
        ours.step()
        still.step()
        assert torch.equal(p, q), step
        gone = weakref.ref(p.grad)
        ours.zero_grad(set_to_none=True)
        assert gone() is None
    p.grad = draw()
    ours.step()
    p.grad = p.grad.t()   # the same address and size, another order
    with pytest.raises(ValueError, match="contiguous"):
        ours.step()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_outlives_moved_gradients(I8, bits):
    """A graph's replay works on the tensors of its capture after eager steps with other gradients."""
    g = torch.Generator().manual_seed(11)
    p, q = (torch.nn.Parameter(torch.ones(3000, device="cuda:0")) for _ in range(2))
    ours, ref = I8.AdamW([p], state_bits=bits), I8.AdamW([q], state_bits=bits)
    fixed = torch.randn(3000, generator=g).cuda()
    q.grad = torch.empty_like(q)

    def twin(grad, number):
        q.grad.copy_(grad)
        if number > 1:
            ref.state[q]["step"] = number - 1
        ref.step()
        torch.cuda.synchronize()
        assert torch.equal(p, q), number

    p.grad = fixed
    ours.step()
    twin(fixed, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ours.step()
    graph.replay()
    twin(fixed, 2)
    for number in (3, 4):
        new = torch.randn(3000, generator=g).cuda()
        p.grad = new.clone()
        ours.step()
        twin(new, number)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda:0") for n in (512, 1024, 4096)]
        graph.replay()
        twin(fixed, 2)
        del junk
