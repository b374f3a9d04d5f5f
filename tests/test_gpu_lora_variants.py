"""The adapters' kernels in every form that the dispatch takes, against the plain
64-bit forms (tests/_finetune.py derives each element's bound), which run on the
GPU here: the forward in one launch, in two with tiles of 16 tokens and with long
tiles, with whole groups of 64 (fp32 32) columns and a whole rank and without, in
every rank class; the gradient's two passes with wide and narrow slices, a
workgroup a tile and blocks of tiles, in every rank class, rows sorted by adapter
and not. A kernel trace of this file names every k_lora_* kernel of the library."""
import pytest
import torch

from tests import _finetune as F
from tests.test_gpu_lora import I8  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
DTS = ["bf16", "f16", "f32"]
CLASSES = [16, 32, 64, 128]


def inputs(dt, T, K, N, R, n, seed):
    """As lora_inputs, made on the GPU."""
    g = torch.Generator(device="cuda:0").manual_seed(seed)

    def randn(shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda:0") * scale).to(F.DT[dt])

    X = randn((T, K))
    X[:, seed % K] *= 20
    return dict(X=X, A=randn((n, R, K), K ** -0.5), B=randn((n, N, R), 0.3),
                scaling=torch.rand(n, generator=g, device="cuda:0") + 0.5, base=randn((T, N)), G=randn((T, N), 0.1),
                base_grad=randn((T, K), 0.1))


def within(got, want, lim, what):
    err = (got.double() - want).abs()
    bad = ~(err <= lim)
    if bad.any():
        i = int(torch.where(bad.view(-1), (err / lim.clamp(min=1e-300)).view(-1).nan_to_num(1e30, 1e30), 0.0).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} beyond their bound; worst at flat {i}: got "
                             f"{got.view(-1)[i].item()!r}, want {want.view(-1)[i].item()!r}, bound "
                             f"{lim.view(-1)[i].item():.3g}")


def segments(T, S, n, seed):
    """S segments of very different lengths, some empty, some without an adapter."""
    g = torch.Generator().manual_seed(seed)
    off = [0] + torch.randint(0, T + 1, (S - 1,), generator=g).sort().values.tolist() + [T]
    return off, torch.randint(-1, n, (S,), generator=g).tolist()


def check(I8, dt, T, K, N, R, n, off, ids, backward, seed=2, with_base=True):  # noqa: F811
    what = f"[{dt} T={T} K={K} N={N} R={R} n={n} S={len(off) - 1}]"
    print("\n  " + what, flush=True)
    c = inputs(dt, T, K, N, R, n, seed)
    segs = F.segments_of(off, ids, n, T)
    so, si = (torch.tensor(x, dtype=torch.int32, device="cuda:0") for x in (off, ids))
    out, V = I8.lora_forward(c["X"], c["A"], c["B"], c["scaling"], so, si, base=c["base"] if with_base else None,
                             with_v=True)
    torch.cuda.synchronize()
    with torch.device("cuda:0"):
        y, lim, v64, vlim = F.lora_forward64(c, dt, segs, with_base)
    within(V, v64, vlim, what + " V")
    within(out, y, lim, what + " out")
    if not backward:
        return
    del y, lim, v64, vlim
    got = I8.lora_backward(c["G"], c["X"], V, c["A"], c["B"], c["scaling"], so, si,
                           base_grad=c["base_grad"] if with_base else None)
    torch.cuda.synchronize()
    with torch.device("cuda:0"):
        want = F.lora_backward64(c, dt, segs, with_base)
    for name, t, (g, e) in zip(("grad_X", "grad_A", "grad_B"), got, want):
        within(t, g, e, f"{what} {name}")


# whole groups of columns and a whole rank, then each of the two broken
COLUMNS = {"whole": (192, 0), "odd width": (200, 0), "odd rank": (192, 7)}
# rows, segments, features of A's rows (over 81920 values of A, or over 32 tiles: two launches)
FORMS = {"one token": (1, 1, lambda R: 320), "tokens in one launch": (24, 24, lambda R: 264),
         "rows in one launch": (90, 4, lambda R: 500), "tokens": (64, 64, lambda R: 260),
         "rows": (40, 3, lambda R: 131072 // R), "long": (1100, 3, lambda R: 520)}


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("R", CLASSES)
@pytest.mark.parametrize("columns", list(COLUMNS))
@pytest.mark.parametrize("form", list(FORMS))
def test_forward(I8, dt, R, columns, form):  # noqa: F811
    T, S, features = FORMS[form]
    N, less = COLUMNS[columns]
    n = min(S, 5)
    if S == T:
        off, ids = list(range(T + 1)), [(3 * i) % n if i % 7 != 5 else -1 for i in range(S)]
    else:
        off, ids = segments(T, S, n, R)
        ids[0], ids[-1] = 0, n - 1
    check(I8, dt, T, features(R), N, R - less, n, off, ids, False, with_base=columns != "odd width")


# rows, columns of the narrow side, segments, adapters: wide slices need (columns / slice) x (rows / 64) of 256 or
# more, blocks of tiles several segments in a block
PASSES = {"wide": (2048, 4096, 3, 2), "wide blocks": (4096, 4096, 40, 40), "wide sorted blocks": (4096, 4096, 200, 40),
          "narrow": (300, 520, 3, 2), "narrow blocks": (6400, 1024, 60, 3), "narrow sorted": (3000, 1000, 300, 5),
          "few sorted": (700, 4096, 50, 1)}


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("R", CLASSES)
@pytest.mark.parametrize("less", [0, 7])
@pytest.mark.parametrize("name", list(PASSES))
def test_backward(I8, dt, R, less, name):  # noqa: F811
    T, C, S, n = PASSES[name]
    off, ids = segments(T, S, n, R + less)
    K, N = C, C
    if R == 16 and "wide" in name and "blocks" in name:
        T = 2 * T                       # two workgroups a unit: blocks of 128 tokens are twice as many
        off = [2 * o for o in off]
    if name.startswith("wide") and R == 32:
        N = 2 * C                       # its wide slices of G are 1024 columns
    if less:
        K, N = K - 3, N - 8             # rows that end inside a slice, of any alignment
    check(I8, dt, T, K, N, R - less, n, off, ids, True, with_base=less == 0)


def test_each_gradient_against_differences(I8):  # noqa: F811
    """fp32: the loss sum(G out) is linear in every single value of X, A and B, so a central difference of the forward
    kernel is the gradient up to the outputs' own error, seen through G; a hundredth of the gradient's median here."""
    T, K, N, R, n = 12, 16, 10, 3, 2
    c = F.lora_inputs("f32", T, K, N, R, n, 25)
    segs = F.segments_of([0, 5, 12], [1, 0], n, T)
    off, ids = (torch.tensor(x, dtype=torch.int32, device="cuda:0") for x in ([0, 5, 12], [1, 0]))
    G = c["G"].double()

    def loss(c):
        """The loss of the kernel's outputs, and how far they may bring it off."""
        out = I8.lora_forward(*(c[k].cuda() for k in ("X", "A", "B", "scaling")), off, ids)
        return float((out.cpu().double() * G).sum()), float((F.lora_forward64(c, "f32", segs, False)[1] * G.abs()).sum())

    d = {k: v.cuda() for k, v in c.items()}
    _, V = I8.lora_forward(d["X"], d["A"], d["B"], d["scaling"], off, ids, with_v=True)
    grads = I8.lora_backward(d["G"], d["X"], V, d["A"], d["B"], d["scaling"], off, ids)
    for name, g, (_, own) in zip("XAB", grads, F.lora_backward64(c, "f32", segs, False)):
        g, h, lims = g.cpu().double(), 0.5, []
        for i in range(g.numel()):
            e = dict(c)
            e[name] = c[name].clone()
            e[name].view(-1)[i] += h
            (up, eu), hi = loss(e), float(e[name].view(-1)[i])
            e[name].view(-1)[i] -= 2 * h
            (dn, ed), lo = loss(e), float(e[name].view(-1)[i])
            lims.append((eu + ed) / (hi - lo) + float(own.view(-1)[i]))
            assert abs((up - dn) / (hi - lo) - float(g.view(-1)[i])) <= lims[-1], (name, i)
        assert max(lims) < 0.01 * float(g[g != 0].abs().median()), (name, max(lims))
