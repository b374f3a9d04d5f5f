"""GPU parity of the adapters beside a shared projection against the plain
64-bit forms (tests/_finetune.py, which derives each element's bound), and of
the autograd function and module against the calls they are made of."""
import pytest
import torch

from tests import _finetune as F

pytestmark = pytest.mark.gpu
DTS = ["bf16", "f16", "f32"]
KEYS = ("X", "A", "B", "scaling", "base", "G", "base_grad")


@pytest.fixture(scope="module")
def I8():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import int8_quantized_linear_rowwise_amd as I8
    return I8


def gpu(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda:0") if isinstance(x, (list, tuple)) else \
        x if x is None else x.cuda()


def check(I8, dt, T, K, N, R, n, off=None, ids=None, seed=1, with_base=True, what=""):
    what = f"[{what} {dt} T={T} K={K} N={N} R={R} n={n}]"
    print("\n  " + what, flush=True)
    c = F.lora_inputs(dt, T, K, N, R, n, seed)
    segs = F.segments_of(off, ids, n, T)
    d = {k: gpu(c[k]) for k in KEYS}
    so, si = gpu(off), gpu(ids)
    out, V = I8.lora_forward(d["X"], d["A"], d["B"], d["scaling"], so, si, base=d["base"] if with_base else None,
                             with_v=True)
    torch.cuda.synchronize()
    y, lim, v64, vlim = F.lora_forward64(c, dt, segs, with_base)
    F.assert_within(V, v64, vlim, what + " V")
    F.assert_within(out, y, lim, what + " out")
    got = I8.lora_backward(d["G"], d["X"], V, d["A"], d["B"], d["scaling"], so, si,
                           base_grad=d["base_grad"] if with_base else None)
    torch.cuda.synchronize()
    for name, t, (g, e) in zip(("grad_X", "grad_A", "grad_B"), got, F.lora_backward64(c, dt, segs, with_base)):
        F.assert_within(t, g, e, f"{what} {name}")


# T, K, N, R, n: from one value to sizes over several tiles, odd and even, every rank class
SIZES = [(1, 1, 1, 1, 1), (3, 7, 5, 2, 1), (1, 512, 264, 16, 1), (17, 64, 40, 16, 1), (33, 72, 136, 8, 1),
         (130, 200, 264, 8, 1), (64, 1040, 520, 64, 1), (100, 264, 328, 128, 1), (70, 131, 77, 100, 1),
         (65, 97, 203, 5, 1), (300, 520, 1032, 32, 1), (257, 1000, 600, 24, 1), (40, 48, 2056, 33, 1),
         (50, 4104, 16, 4, 1)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("T,K,N,R,n", SIZES)
def test_sizes(I8, dt, T, K, N, R, n):
    check(I8, dt, T, K, N, R, n, what="one segment")


SEGMENTS = {
    "a token each": (9, [0, 1, 2, 3, 4, 5, 6, 7, 8, 9], [2, 0, 1, 1, -1, 2, 5, 0, 2]),
    "empty segments": (50, [0, 0, 0, 20, 20, 50, 50], [1, 0, 2, 1, 0, 2]),
    "only empty but one": (16, [0, 0, 16, 16], [0, 1, 2]),
    "none at all": (40, [0, 13, 40], [-1, 7]),
    "no segments": (20, [0], []),
    "borders inside tiles": (200, [0, 15, 16, 17, 63, 64, 65, 129, 200], [0, 1, 2, 0, 1, 2, 0, 1]),
    "one adapter twice": (150, [0, 70, 90, 150], [1, 0, 1]),
    "the identity": (30, [0, 10, 20, 30], None),
    "more segments than rows": (3, [0, 0, 1, 1, 1, 2, 2, 3, 3, 3], [0, 1, 2, 0, 1, 2, 0, 1, 2]),
    "ends not at 0 and T": (25, [4, 10, 20], [0, 1]),
}


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("name", list(SEGMENTS))
def test_segments(I8, dt, name):
    T, off, ids = SEGMENTS[name]
    check(I8, dt, T, 136, 200, 16, 3, off, ids, what=name)


@pytest.mark.parametrize("dt", DTS)
def test_many_segments(I8, dt):
    """More segments than one search step of 64 resolves, most of them short, some empty."""
    g = torch.Generator().manual_seed(3)
    T, S, n = 3000, 5000, 5
    off = [0] + torch.randint(0, T + 1, (S - 1,), generator=g).sort().values.tolist() + [T]
    ids = torch.randint(-1, n, (S,), generator=g).tolist()
    check(I8, dt, T, 40, 24, 4, n, off, ids, what="many segments")


@pytest.mark.parametrize("dt", DTS)
def test_more_adapters_than_segments(I8, dt):
    """Over 64 segments that are not sorted by adapter, as there are as many adapters; most adapters without rows."""
    g = torch.Generator().manual_seed(4)
    T, S, n = 400, 100, 130
    off = [0] + torch.randint(0, T + 1, (S - 1,), generator=g).sort().values.tolist() + [T]
    check(I8, dt, T, 72, 40, 8, n, off, torch.randint(0, n, (S,), generator=g).tolist(), what="many adapters")


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("R", [16, 32])
def test_blocks_of_many_tiles(I8, dt, R):
    """Long batches of many short segments: a workgroup walks the tiles of its block of tokens, segments end inside
    and on the blocks' borders (multiples of 32), and some are empty or without an adapter."""
    g = torch.Generator().manual_seed(5)
    T, S, n = 6000, 40, 4
    off = [0] + torch.randint(0, T + 1, (S - 1,), generator=g).sort().values.tolist() + [T]
    off[10], off[20], off[21] = off[10] // 96 * 96, off[20] // 32 * 32, off[20] // 32 * 32
    off = sorted(off)
    check(I8, dt, T, 1024, 4096, R, n, off, torch.randint(-1, n, (S,), generator=g).tolist(), what="blocks")


@pytest.mark.parametrize("dt", DTS)
def test_without_base(I8, dt):
    check(I8, dt, 90, 264, 136, 16, 2, [0, 40, 90], [1, 0], with_base=False, what="no base")


@pytest.mark.parametrize("dt", DTS)
def test_no_rows_and_no_adapters(I8, dt):
    t = F.DT[dt]
    c = {k: gpu(v) for k, v in F.lora_inputs(dt, 5, 24, 16, 4, 2, 8).items()}
    E = {k: c[k][:0] for k in ("X", "G", "base", "base_grad")}
    out, V = I8.lora_forward(E["X"], c["A"], c["B"], c["scaling"], base=E["base"], with_v=True)
    assert out.shape == (0, 16) and V.shape == (0, 4)
    gA, gB = torch.full_like(c["A"], 7), torch.full_like(c["B"], 7)
    gX, _, _ = I8.lora_backward(E["G"], E["X"], V, c["A"], c["B"], c["scaling"], grad_A=gA, grad_B=gB)
    torch.cuda.synchronize()
    assert gX.shape == (0, 24) and not gA.any() and not gB.any()
    A0, B0, s0 = c["A"][:0], c["B"][:0], c["scaling"][:0]
    out, V = I8.lora_forward(c["X"], A0, B0, s0, base=c["base"], with_v=True)
    assert torch.equal(out, c["base"]) and not V.any()
    gX, gA, gB = I8.lora_backward(c["G"], c["X"], V, A0, B0, s0, base_grad=c["base_grad"])
    assert torch.equal(gX, c["base_grad"]) and gA.shape == (0, 4, 24) and gB.shape == (0, 16, 4)
    # rank 0 and empty widths
    out = I8.lora_forward(c["X"], torch.empty(2, 0, 24, dtype=t, device="cuda:0"),
                          torch.empty(2, 16, 0, dtype=t, device="cuda:0"), c["scaling"], base=c["base"])
    assert torch.equal(out, c["base"])
    out = I8.lora_forward(c["X"][:, :0], c["A"][:, :, :0], c["B"], c["scaling"], base=c["base"])
    assert torch.equal(out, c["base"])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_second_part_of_v_counts(I8, dt):
    """base takes away the rounded product, so what is left is far below one step of the output's type: V has to
    enter the product with its 16 bits."""
    T, K, N, R = 40, 32, 136, 16
    c = F.lora_inputs(dt, T, K, N, R, 1, 5)
    y, _, _, _ = F.lora_forward64(c, dt, [(0, T, 0)], with_base=False)
    c["base"] = (-y).to(F.DT[dt])
    y, lim, _, _ = F.lora_forward64(c, dt, [(0, T, 0)])
    out = I8.lora_forward(*(gpu(c[k]) for k in ("X", "A", "B", "scaling")), base=gpu(c["base"]))
    F.assert_within(out, y, lim, "remainder")


@pytest.mark.parametrize("scale", [1e-7, 1e6])
def test_f16_range_of_v(I8, scale):
    """V far below fp16's smallest or above its largest value: fp32 V takes part in full."""
    T, K, N, R = 70, 64, 72, 16
    c = F.lora_inputs("f16", T, K, N, R, 2, 6)
    up = min(scale, 1.0)
    c["A"] = (c["A"].double() * (100.0 if scale > 1 else up)).to(torch.float16)
    c["X"] = (c["X"].double() * (200.0 if scale > 1 else 1.0)).clamp(-6e4, 6e4).to(torch.float16)
    c["B"] = (c["B"].double() * (1e-3 if scale > 1 else 10.0)).to(torch.float16)
    c["scaling"] = c["scaling"] * (1e-3 if scale > 1 else 1e5)
    segs = [(0, 30, 0), (30, 70, 1)]
    d = {k: gpu(c[k]) for k in KEYS}
    off = gpu([0, 30, 70])
    out, V = I8.lora_forward(d["X"], d["A"], d["B"], d["scaling"], off, base=d["base"], with_v=True)
    y, lim, v64, vlim = F.lora_forward64(c, "f16", segs)
    assert (v64.abs().max() > 65504) == (scale > 1)
    F.assert_within(V, v64, vlim, "V")
    F.assert_within(out, y, lim, "out")
    got = I8.lora_backward(d["G"], d["X"], V, d["A"], d["B"], d["scaling"], off, base_grad=d["base_grad"])
    for name, t, (g, e) in zip(("grad_X", "grad_A", "grad_B"), got, F.lora_backward64(c, "f16", segs)):
        over = g.abs() + e >= 65504
        F.assert_within(torch.where(over, 0.0, t.cpu().double()), torch.where(over, 0.0, g), e, name)


@pytest.mark.parametrize("dt", DTS)
def test_values_that_are_not_finite_stay_in_their_rows(I8, dt):
    """An infinity or NaN in one row (also one without an adapter) reaches no other row's output."""
    T, K, N, R = 40, 72, 40, 8
    c = F.lora_inputs(dt, T, K, N, R, 2, 9)
    off, ids = [0, 10, 12, 40], [0, -1, 1]
    ref = {k: gpu(c[k].clone()) for k in KEYS}
    args = lambda d: (d["A"], d["B"], d["scaling"], gpu(off), gpu(ids))  # noqa: E731
    want, V0 = I8.lora_forward(ref["X"], *args(ref), base=ref["base"], with_v=True)
    bad = {k: v.clone() for k, v in ref.items()}
    bad["X"][11, 3], bad["X"][20, 5], bad["base"][30, 7] = float("nan"), float("inf"), float("nan")
    out, V = I8.lora_forward(bad["X"], *args(bad), base=bad["base"], with_v=True)
    torch.cuda.synchronize()
    keep = [t for t in range(T) if t not in (20, 30)]
    assert torch.equal(out[keep], want[keep]) and not torch.isfinite(out[20]).any()
    assert torch.isnan(out[30, 7]) and torch.equal(out[30, :7], want[30, :7])
    assert torch.equal(V[keep], V0[keep])
    # gradients: the rows without an adapter take part in none
    w = I8.lora_backward(ref["G"], ref["X"], V0, *args(ref), base_grad=ref["base_grad"])
    bad = {k: v.clone() for k, v in ref.items()}
    bad["X"][11], bad["G"][10] = float("nan"), float("inf")
    g = I8.lora_backward(bad["G"], bad["X"], V0, *args(bad), base_grad=bad["base_grad"])
    torch.cuda.synchronize()
    for a, b, name in zip(g, w, ("grad_X", "grad_A", "grad_B")):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("dt", DTS)
def test_offsets_that_make_no_sense_stay_inside(I8, dt):
    """Offsets out of range or order: no row outside the tensors is read or written (the rows around the output keep
    their values), and the next call is right."""
    T, K, N, R, n = 50, 72, 40, 8, 2
    c = {k: gpu(v) for k, v in F.lora_inputs(dt, T, K, N, R, n, 10).items()}
    frame = torch.full((T + 200, N), 3.0, dtype=F.DT[dt], device="cuda:0")
    gframe = torch.full((T + 200, K), 3.0, dtype=F.DT[dt], device="cuda:0")
    V = torch.zeros(T, R, device="cuda:0")
    for off, ids in (([0, 1 << 30, -5, 50], [0, 1, 1]), ([50, 40, 30, 0], [0, 1, -9]), ([-(1 << 31), 60, 70, 80],
                                                                                       [0, (1 << 31) - 1, 1])):
        I8.lora_forward(c["X"], c["A"], c["B"], c["scaling"], gpu(off), gpu(ids), base=c["base"],
                        out=frame[100:100 + T])
        I8.lora_backward(c["G"], c["X"], V, c["A"], c["B"], c["scaling"], gpu(off), gpu(ids),
                         grad_X=gframe[100:100 + T])
        torch.cuda.synchronize()
        for f in (frame, gframe):
            assert (f[:100] == 3).all() and (f[100 + T:] == 3).all()
    check(I8, dt, T, K, N, R, n, [0, 20, 50], [1, 0], what="afterwards")


@pytest.mark.parametrize("dt", DTS)
def test_in_place_and_parts(I8, dt):
    """out = base and grad_X = base_grad give the same bits, as do calls for one gradient alone."""
    T, K, N, R, n = 150, 264, 328, 16, 2
    c = {k: gpu(v) for k, v in F.lora_inputs(dt, T, K, N, R, n, 11).items()}
    args = (c["A"], c["B"], c["scaling"], gpu([0, 70, 150]), gpu([1, 0]))
    out, V = I8.lora_forward(c["X"], *args, base=c["base"], with_v=True)
    y = c["base"].clone()
    assert I8.lora_forward(c["X"], *args, base=y, out=y) is y and torch.equal(y, out)
    gX, gA, gB = I8.lora_backward(c["G"], c["X"], V, *args, base_grad=c["base_grad"])
    y = c["base_grad"].clone()
    I8.lora_backward(c["G"], c["X"], V, *args, base_grad=y, grad_X=y)
    assert torch.equal(y, gX)
    for i, want in enumerate((gX, gA, gB)):
        on = [j == i for j in range(3)]
        got = I8.lora_backward(c["G"], c["X"], V, *args, base_grad=c["base_grad"], with_grad_X=on[0],
                               with_grad_A=on[1], with_grad_B=on[2])
        assert torch.equal(got[i], want) and all(got[j] is None for j in range(3) if j != i)


@pytest.mark.parametrize("dt", DTS)
def test_unaligned_views(I8, dt):
    """Contiguous views that start one element into their storage give the results of aligned copies."""
    T, K, N, R, n = 70, 264, 136, 16, 2
    c = {k: gpu(v) for k, v in F.lora_inputs(dt, T, K, N, R, n, 12).items()}

    def shift(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        s[1:] = t.reshape(-1)
        return s[1:].view(t.shape)

    off, ids = gpu([0, 30, 70]), gpu([1, 0])
    want, V = I8.lora_forward(c["X"], c["A"], c["B"], c["scaling"], off, ids, base=c["base"], with_v=True)
    wg = I8.lora_backward(c["G"], c["X"], V, c["A"], c["B"], c["scaling"], off, ids, base_grad=c["base_grad"])
    s = {k: shift(v) for k, v in c.items()}
    out = I8.lora_forward(s["X"], s["A"], s["B"], s["scaling"], off, ids, base=s["base"],
                          out=shift(torch.zeros_like(want)))
    gg = I8.lora_backward(s["G"], s["X"], shift(V), s["A"], s["B"], s["scaling"], off, ids, base_grad=s["base_grad"],
                          grad_X=shift(c["X"]), grad_A=shift(c["A"]), grad_B=shift(c["B"]))
    ref = {k: v.cpu() for k, v in c.items()}
    segs = F.segments_of([0, 30, 70], [1, 0], n, T)
    y, lim, _, _ = F.lora_forward64(ref, dt, segs)
    F.assert_within(out, y, lim, "shifted out")
    for name, t, (g, e) in zip(("grad_X", "grad_A", "grad_B"), gg, F.lora_backward64(ref, dt, segs)):
        F.assert_within(t, g, e, "shifted " + name)
    assert len(wg) == 3


@pytest.mark.parametrize("dt", DTS)
def test_deterministic(I8, dt):
    T, K, N, R, n = 700, 1032, 520, 16, 3
    c = {k: gpu(v) for k, v in F.lora_inputs(dt, T, K, N, R, n, 13).items()}
    args = (c["A"], c["B"], c["scaling"], gpu([0, 100, 101, 400, 700]), gpu([1, 0, 2, 1]))
    first = None
    for _ in range(4):
        out, V = I8.lora_forward(c["X"], *args, base=c["base"], with_v=True)
        r = (out, V) + I8.lora_backward(c["G"], c["X"], V, *args, base_grad=c["base_grad"])
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(r, first))
        first = r


@pytest.mark.parametrize("dt", ["bf16"])
@pytest.mark.parametrize("shape", ["wide", "long"])
def test_layer_sizes_sampled(I8, dt, shape):
    """The 7B block's up projection with 4096 tokens, and a long batch: sampled rows and columns against 64 bits."""
    T, K, N, R, n, off, ids = {"wide": (4096, 4096, 11008, 16, 2, [0, 1500, 2048, 4096], [1, -1, 0]),
                               "long": (20011, 1024, 1032, 64, 3, [0, 7000, 7001, 15000, 20011], [2, 0, 1, 2])}[shape]
    print(f"\n  [{shape}]", flush=True)
    c = F.lora_inputs(dt, T, K, N, R, n, 14)
    d = {k: gpu(v) for k, v in c.items()}
    args = (d["A"], d["B"], d["scaling"], gpu(off), gpu(ids))
    out, V = I8.lora_forward(d["X"], *args, base=d["base"], with_v=True)
    gX, gA, gB = I8.lora_backward(d["G"], d["X"], V, *args, base_grad=d["base_grad"])
    torch.cuda.synchronize()
    g = torch.Generator().manual_seed(1)
    rows = torch.unique(torch.cat([torch.tensor([0, T - 1] + [o for o in off if o < T] + [o - 1 for o in off if o > 0]),
                                   torch.randint(0, T, (150,), generator=g)]))
    segs = F.segments_of(off, ids, n, T)
    own = torch.full((T,), -1)
    for lo, hi, a in segs:
        own[lo:hi] = a
    few = dict(c, X=c["X"][rows], base=c["base"][rows], G=c["G"][rows], base_grad=c["base_grad"][rows])
    s = [(i, i + 1, int(own[t])) for i, t in enumerate(rows)]
    y, lim, v64, vlim = F.lora_forward64(few, dt, s)
    F.assert_within(out[rows.cuda()], y, lim, "out")
    F.assert_within(V[rows.cuda()], v64, vlim, "V")
    (wX, eX), _, _ = F.lora_backward64(few, dt, s)
    F.assert_within(gX[rows.cuda()], wX, eX, "grad_X")
    # grad_A at some input features, grad_B at some output features; the other operand is whole
    ks = torch.unique(torch.cat([torch.tensor([0, K - 1]), torch.randint(0, K, (30,), generator=g)]))
    ns = torch.unique(torch.cat([torch.tensor([0, N - 1]), torch.randint(0, N, (30,), generator=g)]))
    U, D = F.U, F.D
    for a in range(n):
        rows = own == a
        x, gg, A, B, f = c["X"][rows].to(D), c["G"][rows].to(D), c["A"][a].to(D), c["B"][a].to(D), c["scaling"][a].to(D)
        m = x.shape[0]
        dV, eV = f * (gg @ B), 1.01 * (N + 2) * U * f * (gg.abs() @ B.abs())
        want = dV.t() @ x[:, ks]
        e = eV.t() @ x[:, ks].abs() + (2.0 ** -17 + 1.01 * (2 * m + 4) * U) * ((dV.abs() + eV).t() @ x[:, ks].abs())
        F.assert_within(gA[a][:, ks.cuda()], want, e + (want.abs() + e) * F.half_step(dt), f"grad_A {a}")
        v, ev = x @ A.t(), 1.01 * K * U * (x.abs() @ A.abs().t())
        want = f * (gg[:, ns].t() @ v)
        e = f * (gg[:, ns].abs().t() @ (ev + (2.0 ** -17 + 1.01 * (2 * m + 4) * U) * (v.abs() + ev)))
        F.assert_within(gB[a][ns.cuda()], want, e + (want.abs() + e) * F.half_step(dt), f"grad_B {a}")


def test_rows_past_32_bit_offsets(I8):
    """More than 2^31 elements in X and out: the last rows are right."""
    T, K, N, R = (1 << 18) + 5, 8200, 8, 1
    X = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda:0")
    X[-3:] = F.randn((3, K), "bf16", 1).cuda()
    c = F.lora_inputs("bf16", 3, K, N, R, 1, 2)
    c["X"] = X[-3:].cpu()
    base = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda:0")
    base[-3:] = c["base"].cuda()
    out, V = I8.lora_forward(X, gpu(c["A"]), gpu(c["B"]), gpu(c["scaling"]), base=base, with_v=True)
    y, lim, v64, vlim = F.lora_forward64(c, "bf16", [(0, 3, 0)])
    F.assert_within(out[-3:], y, lim, "out")
    F.assert_within(V[-3:], v64, vlim, "V")
    assert not out[:-3].any()
    G = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda:0")
    G[-3:] = c["G"].cuda()
    gX, gA, gB = I8.lora_backward(G, X, V, gpu(c["A"]), gpu(c["B"]), gpu(c["scaling"]))
    w = F.lora_backward64(c, "bf16", [(0, 3, 0)], with_base=False)
    F.assert_within(gX[-3:], *w[0], "grad_X")
    assert not gX[:-3].any()
    F.assert_within(gA, *w[1], "grad_A")
    F.assert_within(gB, *w[2], "grad_B")


def test_side_stream_and_graph(I8):
    T, K, N, R, n = 200, 520, 264, 16, 3
    mk = lambda seed: {k: gpu(v) for k, v in F.lora_inputs("bf16", T, K, N, R, n, seed).items()}  # noqa: E731
    c = mk(15)
    off, ids = gpu([0, 60, 61, 200]), gpu([2, 0, 1])

    def calls(c):
        out, V = I8.lora_forward(c["X"], c["A"], c["B"], c["scaling"], off, ids, base=c["base"], with_v=True)
        return (out, V) + I8.lora_backward(c["G"], c["X"], V, c["A"], c["B"], c["scaling"], off, ids,
                                           base_grad=c["base_grad"])

    want = calls(c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = calls(c)
    calls(mk(16))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = calls(c)
    for seed in (17, 18, 19):
        new = mk(seed)
        for k in KEYS:
            c[k].copy_(new[k])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, calls(new))), seed


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_autograd_function_and_module(I8, dt):
    """The module's output and gradients are the calls' bits: int8 layer, then the adapters in place; gradients of a
    batch that uses one adapter twice; and a module without segments uses adapter 0."""
    M, K, N, n, R = 96, 264, 136, 3, 8
    W = F.randn((N, K), "f32", 20, 0.05).cuda()
    lin = I8.Int8LoraLinear(W, F.randn((N,), "f32", 21).cuda(), adapters=n, rank=R, alpha=12.0, dtype=F.DT[dt])
    with torch.no_grad():
        lin.lora_B.copy_(F.randn((n, N, R), dt, 22, 0.1))
    x = F.randn((2, M // 2, K), dt, 23).cuda().requires_grad_(True)
    off, ids = gpu([0, 30, 60, 96]), gpu([1, 2, 1])
    y = lin(x, off, ids)
    g = F.randn((2, M // 2, N), dt, 24, 0.1).cuda()
    y.backward(g)
    X, G = x.detach().reshape(M, K), g.reshape(M, N)
    b = lin.bias.detach().to(x.dtype)
    base = I8.int8_linear_forward(X, lin.CB, lin.SCB, b, 6.0)
    A, B = lin.lora_A.detach(), lin.lora_B.detach()
    out, V = I8.lora_forward(X, A, B, lin.scaling, off, ids, base=base, with_v=True)
    bg, gb = I8.int8_linear_backward_input(G, lin.CB, lin.SCB)
    gX, gA, gB = I8.lora_backward(G, X, V, A, B, lin.scaling, off, ids, base_grad=bg)
    assert torch.equal(y.detach().reshape(M, N), out) and torch.equal(x.grad.reshape(M, K), gX)
    assert torch.equal(lin.lora_A.grad, gA) and torch.equal(lin.lora_B.grad, gB)
    assert torch.equal(lin.bias.grad, gb.float()) and not lin.lora_A.grad[0].any()
    one = I8.lora_forward(X, A, B, lin.scaling, gpu([0, M]), gpu([0]), base=base)
    assert torch.equal(lin(x.detach()).reshape(M, N), one)


def test_gradients_against_differences(I8):
    """fp32: the backward's gradients against central differences of the forward kernel (the loss is a product of
    three factors, so a difference over 2 h is exact but for fp32's rounding of the outputs)."""
    T, K, N, R, n = 12, 16, 10, 3, 2
    c = {k: gpu(v) for k, v in F.lora_inputs("f32", T, K, N, R, n, 25).items()}
    off, ids = gpu([0, 5, 12]), gpu([1, 0])

    def loss(c):
        out = I8.lora_forward(c["X"], c["A"], c["B"], c["scaling"], off, ids)
        return float((out.double() * c["G"].double()).sum())

    _, V = I8.lora_forward(c["X"], c["A"], c["B"], c["scaling"], off, ids, with_v=True)
    grads = dict(zip("XAB", I8.lora_backward(c["G"], c["X"], V, c["A"], c["B"], c["scaling"], off, ids)))
    out = I8.lora_forward(c["X"], c["A"], c["B"], c["scaling"], off, ids)
    h = 2.0 ** -4
    # outputs are off by at most (K + 2 R + 6) u times a few of their own size each, seen through G
    lim = 4 * (K + 2 * R + 6) * F.U * float((out.double().abs() * c["G"].double().abs()).sum() * 20) / h
    for name, g in grads.items():
        for i in range(0, g.numel(), 3):
            d = dict(c)
            d[name] = c[name].clone()
            d[name].view(-1)[i] += h
            up, hi = loss(d), float(d[name].view(-1)[i])
            d[name].view(-1)[i] -= 2 * h
            lo = float(d[name].view(-1)[i])
            assert abs((up - loss(d)) / (hi - lo) - float(g.view(-1)[i])) <= lim, (name, i)
