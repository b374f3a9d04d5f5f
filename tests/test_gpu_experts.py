"""The experts' operators on the GPU against their plain 64-bit forms (tests/_experts.py)."""
import pytest
import torch

from tests import _experts as X
from tests._gpu import TORCH

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def I8():
    import int8_quantized_linear_rowwise_amd as m
    return m


def gpu(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


# ---- sort -----------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,E,drop", [
    (1, 2, 8, 0), (0, 2, 4, 0), (5, 0, 4, 0), (3, 1, 1, 0), (7, 3, 0, 0), (64, 4, 64, 0), (257, 2, 5, 0.5),
    (1024, 2, 128, 0), (1025, 2, 128, 0.1), (3000, 8, 1000, 0.1), (2048, 1, 1024, 0), (777, 3, 7, 1.0),
    (5000, 8, 3, 0.02), (8192, 1, 40, 0.1), (4097, 2, 9, 0), (1, 1, 1024, 0), (129, 63, 100, 0.3),
])
def test_sort(I8, T, k, E, drop, dtype):
    ids = X.choices(T, k, E, T + k, drop).to(dtype)
    want = X.sort(ids, E)
    got = I8.expert_sort(ids.to(DEV), E)
    for g, w, what in zip(got, want, ("offsets", "tokens", "positions")):
        assert g.dtype == torch.int32 and torch.equal(g.cpu(), w), what


def test_sort_values_out_of_range(I8):
    ids = torch.tensor([[0, 3], [2 ** 33, -2 ** 40], [2, 2 ** 32 + 1], [4, -1]])
    want = X.sort(ids, 4)
    for g, w in zip(I8.expert_sort(ids.to(DEV), 4), want):
        assert torch.equal(g.cpu(), w)
    low = torch.tensor([[2 ** 31 - 1, -2 ** 31], [1, 0]], dtype=torch.int32)
    for g, w in zip(I8.expert_sort(low.to(DEV), 2), X.sort(low, 2)):
        assert torch.equal(g.cpu(), w)


def test_sort_one_expert_takes_all(I8):
    ids = torch.full((9000, 2), 6)
    for g, w in zip(I8.expert_sort(ids.to(DEV), 9), X.sort(ids, 9)):
        assert torch.equal(g.cpu(), w)


def test_sort_large(I8):
    """More choices than a workgroup's usual share a block: against torch's stable sort."""
    T, k, E = 150001, 8, 37
    g = torch.Generator(device=DEV).manual_seed(5)
    ids = torch.randint(-1, E, (T, k), generator=g, device=DEV)
    off, token, pos = I8.expert_sort(ids, E)
    flat = ids.view(-1)
    by, order = torch.where(flat < 0, E, flat).sort(stable=True)
    n = int((flat >= 0).sum())
    assert torch.equal(off.long(), torch.searchsorted(by, torch.arange(E + 1, device=DEV)))
    assert torch.equal(token[:n].long(), order[:n] // k) and bool((token[n:] == -1).all())
    row = torch.empty_like(flat)
    row[order] = torch.arange(T * k, device=DEV)
    assert torch.equal(pos.view(-1).long(), torch.where(flat < 0, -1, row))


# ---- products -------------------------------------------------------------------------------------------------------


def run_forward(I8, dt, T, K, N, off, ids=None, rows=None, E=None, tau=6.0, outliers=2, seed=1):
    E = len(off) - 1 if E is None else E
    CB, SCB = X.weights(E, N, K, seed)
    x = X.inputs(T, K, dt, seed + 1, outliers)
    off = torch.tensor(off, dtype=torch.int32)
    ids = None if ids is None else torch.tensor(ids, dtype=torch.int32)
    rows = None if rows is None else torch.as_tensor(rows, dtype=torch.int32)
    x, CB, SCB, off, ids, rows = gpu(x, CB, SCB, off, ids, rows)
    got = I8.expert_forward(x, CB, SCB, off, ids, rows, tau)
    y, slack = X.forward(x, CB, SCB, off, ids, rows, tau)
    X.check(got, y, X.rounded(y, slack, dt), "out")
    assert torch.equal(got, I8.expert_forward(x, CB, SCB, off, ids, rows, tau))
    return got


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K,N", [(64, 64), (128, 192), (200, 72), (1001, 530), (16, 8), (1, 1), (4096, 136), (24, 260)])
def test_forward_sizes(I8, dt, K, N):
    run_forward(I8, dt, 45, K, N, [0, 0, 7, 40, 45])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off", [[0, 1], [0, 129, 129, 256, 300], [0] * 40 + [3], [0, 15, 16, 17, 33, 64, 65],
                                 [0, 0, 0]])
def test_forward_segments(I8, dt, off):
    run_forward(I8, dt, max(off[-1], 1), 160, 144, off)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_forward_rows_without_expert_or_token(I8, dt):
    """Unknown experts, unknown tokens and the rows behind the last offset: zeros, whatever lay there."""
    got = run_forward(I8, dt, 10, 96, 80, [0, 3, 6, 9], ids=[1, -1, 5], rows=[9, -1, 0, 1, 2, 3, 4, 5, 6, 7, 8], E=2)
    assert (got[1] == 0).all() and (got[3:] == 0).all() and (got[0] != 0).any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,E,K,N", [(1, 2, 8, 256, 320), (33, 2, 4, 128, 96), (300, 4, 6, 320, 256),
                                          (700, 2, 3, 512, 512)])
def test_forward_sorted(I8, dt, T, k, E, K, N):
    off, token, _ = X.sort(X.choices(T, k, E, 7, 0.1), E)
    run_forward(I8, dt, T, K, N, off.tolist(), rows=token)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("outliers", [0, 1, 15, 16, 17, 64, 65, 100, 300])
def test_forward_outlier_columns(I8, dt, outliers):
    run_forward(I8, dt, 150, 320, 264, [0, 30, 150], outliers=outliers)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,E,K,N,outliers", [(1500, 2, 4, 272, 1100, 3), (1500, 2, 4, 272, 4100, 40),
                                                (800, 2, 3, 64, 3000, 1), (2100, 3, 9, 400, 2304, 17),
                                                (600, 1, 1, 16, 5000, 0), (1500, 2, 4, 271, 1101, 20),
                                                (900, 2, 3, 1001, 530, 3), (700, 1, 2, 17, 4099, 1),
                                                (800, 1, 2, 15, 600, 1), (520, 1, 1, 129, 257, 0)])
def test_forward_many_rows(I8, dt, T, k, E, K, N, outliers):
    """Sizes that fill tiles of 256 rows, with contractions and widths that end inside one, more outlier columns than
    fit beside the tile, and experts of very different numbers of rows."""
    off, token, _ = X.sort(X.choices(T, k, E, 7, 0.1, skew=1.5), E)
    run_forward(I8, dt, T, K, N, off.tolist(), rows=token, outliers=outliers)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,E,K,N,outliers", [(1, 1, 1, 16, 8, 0), (1, 2, 8, 4096, 136, 4), (1, 3, 3, 272, 50, 17),
                                                (2, 2, 5, 2064, 33, 300), (3, 2, 4, 1024, 64, 600),
                                                (4, 2, 4, 4096, 48, 33), (4, 4, 4, 48, 17, 5), (5, 2, 4, 4096, 48, 3),
                                                (4, 1, 2, 4112, 32, 3)])
def test_forward_few_tokens(I8, dt, T, k, E, K, N, outliers):
    """Up to four tokens are quantized in the product's own launch; one more, or one piece more, is not."""
    off, token, _ = X.sort(X.choices(T, k, E, 7, 0.1), E)
    a = run_forward(I8, dt, T, K, N, off.tolist(), rows=token, outliers=outliers)
    run_forward(I8, dt, T, K, N, off.tolist(), rows=token, outliers=outliers, tau=0.0)
    if T == 4:
        # beside a fifth token, with the same outlier columns, the rows are the same
        CB, SCB = gpu(*X.weights(E, N, K, 1))
        x = X.inputs(T, K, dt, 2, outliers).to(DEV)
        five = torch.cat([x, x[:1]])
        off, token = gpu(off, token)
        assert torch.equal(I8.expert_forward(five, CB, SCB, off, rows=token), a)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K,N", [(4, 9), (12, 40), (20, 33), (1004, 31), (4092, 24), (4088, 17)])
@pytest.mark.parametrize("T", [1, 4])
def test_forward_few_tokens_between_borders(I8, dt, T, K, N):
    """Contractions that are whole words and no whole pieces: what follows a row of weights must not reach its sums."""
    off, token, _ = X.sort(X.choices(T, 2, 3, 7, 0.1), 3)
    run_forward(I8, dt, T, K, N, off.tolist(), rows=token)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,E,K,N,shift", [(700, 2, 3, 1040, 512, 0), (1500, 2, 4, 1100, 1100, 4),
                                             (1500, 2, 4, 1041, 4101, 0), (900, 2, 3, 2001, 530, 1),
                                             (2100, 3, 9, 1288, 2304, 0), (600, 1, 1, 1030, 5000, 2),
                                             (300, 1, 2, 1044, 150, 0), (700, 2, 3, 1028, 300, 12)])
def test_forward_long_contractions(I8, dt, T, k, E, K, N, shift):
    """Past what the tiles for short contractions take; weights that begin off a border."""
    off, token, _ = X.sort(X.choices(T, k, E, 7, 0.1, skew=1.5), E)
    CB, SCB = X.weights(E, N, K, 3)
    x, off, token, SCB = gpu(X.inputs(T, K, dt, 4, 5), off, token, SCB)
    place = torch.zeros(E * N * K + 16, dtype=torch.int8, device=DEV)
    CB = place[shift:shift + E * N * K].view(E, N, K).copy_(CB)
    got = I8.expert_forward(x, CB, SCB, off, rows=token)
    y, slack = X.forward(x, CB, SCB, off, None, token, 6.0)
    X.check(got, y, X.rounded(y, slack, dt), "out")


def _codes(*shape):
    g = torch.Generator(device=DEV).manual_seed(5)
    return torch.randint(-127, 128, shape, dtype=torch.int8, device=DEV, generator=g)


@pytest.mark.parametrize("T,E,N,K", [(5, 17, 8192, 16384), (40, 17, 8192, 16384), (600, 17, 8192, 16384),
                                     (600, 600, 8192, 512)])
def test_weights_past_32_bits(I8, T, E, N, K):
    """Weights of over 2^31 bytes: the last expert's products and gradients are those of that expert alone."""
    CB, SCB = _codes(E, N, K), torch.rand((E, N), device=DEV) + 0.5
    x, G = X.inputs(T, K, "bf16", 1).to(DEV), X.inputs(T, N, "bf16", 2, 0).to(DEV)
    for ids in ([E - 1], [0]):
        off, seg = torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.tensor(ids, dtype=torch.int32, device=DEV)
        one = slice(ids[0], ids[0] + 1)
        assert torch.equal(I8.expert_forward(x, CB, SCB, off, seg), I8.expert_forward(x, CB[one], SCB[one], off))
        assert torch.equal(I8.expert_backward(G, CB, SCB, off, seg), I8.expert_backward(G, CB[one], SCB[one], off))


@pytest.mark.parametrize("N", [262144, 262143])
def test_rows_past_32_bits(I8, N):
    """Over 2^31 outputs, and gradients: the last rows are those of a call with these rows alone."""
    T, K, last = 9000, 16, 300
    CB, SCB = _codes(1, N, K), torch.rand((1, N), device=DEV) + 0.5
    x = X.inputs(T, K, "bf16", 1, 0).to(DEV)
    off, few = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (T, last))
    out = I8.expert_forward(x, CB, SCB, off, threshold=0.0)
    assert torch.equal(out[-last:], I8.expert_forward(x[-last:], CB, SCB, few, threshold=0.0))
    g = I8.expert_backward(out, CB, SCB, off)
    assert torch.equal(g[-last:], I8.expert_backward(out[-last:].contiguous(), CB, SCB, few))
    pos = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1)
    assert torch.equal(I8.expert_combine(out, pos[-last:]), out[-last:])
    gY, gg = I8.expert_combine_backward(out, pos, None, out)
    assert torch.equal(gY, out) and bool((gg[-last:] > 0).all())


def test_tokens_past_32_bits(I8):
    """Over 2^31 codes: the last tokens' products are those of these tokens alone."""
    T, K, N, last = 140000, 16384, 256, 700
    x = X.inputs(1000, K, "bf16", 1, 0).to(DEV).repeat(T // 1000, 1)
    x[-last:] *= torch.linspace(0.5, 2.0, last, device=DEV, dtype=torch.bfloat16)[:, None]
    CB, SCB = _codes(2, N, K), torch.rand((2, N), device=DEV) + 0.5
    for n in (12, last):
        off = torch.tensor([0, n // 3, n], dtype=torch.int32, device=DEV)
        rows = torch.arange(T - n, T, dtype=torch.int32, device=DEV).flip(0)
        got = I8.expert_forward(x, CB, SCB, off, rows=rows, threshold=0.0)
        assert torch.equal(got, I8.expert_forward(x[-n:], CB, SCB, off, rows=rows - (T - n), threshold=0.0))


@pytest.mark.parametrize("tau", [0.0, -1.0, float("inf"), float("nan"), 1.0])
def test_forward_thresholds(I8, tau):
    run_forward(I8, "bf16", 20, 128, 64, [0, 8, 20], tau=tau)


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("T,K,N,R", [(2, 64, 40, 9), (40, 64, 40, 60), (700, 64, 3000, 2000), (700, 2048, 600, 1200)])
def test_forward_rows_without_token_hide_weights(I8, dt, T, K, N, R):
    """Rows without a token are zeros even where the expert's scales are not finite, in every kernel."""
    CB, SCB = gpu(*X.weights(2, N, K, 1))
    x = X.inputs(T, K, dt, 2).to(DEV)
    SCB[:, ::3] = float("inf")
    SCB[:, 1::3] = float("nan")
    rows = (torch.arange(R) % T).int()
    rows[::5] = -1
    rows[3::7] = T
    off = torch.tensor([0, R // 3, R], dtype=torch.int32, device=DEV)
    out = I8.expert_forward(x, CB, SCB, off, rows=rows.to(DEV))
    none = ((rows < 0) | (rows >= T)).to(DEV)
    assert (out[none] == 0).all() and (out[~none][:, 1::3]).isnan().all()


def test_forward_more_segments_than_experts(I8):
    """Many short segments that share experts, in any order; over 64 and over 4096 segments."""
    for S in (70, 4500):
        off = [min(i * 2, 900) for i in range(S + 1)]
        run_forward(I8, "f16", 901, 64, 32, off, ids=[(5 * i) % 7 - 1 for i in range(S)], E=5)


def test_forward_empty(I8):
    z = torch.zeros
    CB, SCB = z((2, 6, 8), dtype=torch.int8, device=DEV), z((2, 6), device=DEV)
    off = z(3, dtype=torch.int32, device=DEV)
    assert I8.expert_forward(z((0, 8), device=DEV), CB, SCB, off).shape == (0, 6)
    rows = z(4, dtype=torch.int32, device=DEV)
    out = torch.full((4, 6), 7.0, device=DEV)
    I8.expert_forward(z((0, 8), device=DEV), CB, SCB, off, rows=rows, out=out)           # no tokens
    assert (out == 0).all()
    out.fill_(7)
    I8.expert_forward(z((4, 0), device=DEV), CB[:, :, :0], SCB, off + 4, out=out)        # no features
    assert (out == 0).all()
    out.fill_(7)
    I8.expert_forward(z((4, 8), device=DEV), CB, SCB, off[:1], out=out)                  # no segments
    assert (out == 0).all()
    assert I8.expert_forward(z((4, 8), device=DEV), CB[:, :0], SCB[:, :0], off).shape == (4, 0)


def test_forward_bad_offsets_stay_inside(I8):
    """Offsets that are not non-decreasing or leave [0, R]: undefined rows, but nothing outside `out` is written."""
    R, N = 100, 40
    CB, SCB = gpu(*X.weights(3, N, 64, 1))
    x = X.inputs(R, 64, "bf16", 2).to(DEV)
    pad = torch.full((R + 64, N), 3.0, dtype=torch.bfloat16, device=DEV)
    for off in ([0, 50, 20, 90], [0, -5, 1000, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31, 7, 3], [90, 80, 10, 0]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        I8.expert_forward(x, CB, SCB, o, out=pad[32:32 + R])
        I8.expert_backward(x[:, :N].contiguous(), CB, SCB, o)
        assert (pad[:32] == 3).all() and (pad[32 + R:] == 3).all()


def test_forward_unaligned_tensors(I8):
    """Tensors that start off the 16-byte borders."""
    T, K, N = 21, 64, 40
    CB, SCB = X.weights(2, N, K, 1)
    x = X.inputs(T, K, "f16", 2)
    raw = torch.zeros(T * K + 1, dtype=torch.float16, device=DEV)
    xg = raw[1:].view(T, K).copy_(x)
    rawc = torch.zeros(2 * N * K + 3, dtype=torch.int8, device=DEV)
    cg = rawc[3:].view(2, N, K).copy_(CB)
    outr = torch.zeros(T * N + 1, dtype=torch.float16, device=DEV)
    off = torch.tensor([0, 5, T], dtype=torch.int32, device=DEV)
    I8.expert_forward(xg, cg, SCB.to(DEV), off, out=outr[1:].view(T, N))
    y, slack = X.forward(x, CB, SCB, off.cpu())
    X.check(outr[1:].view(T, N).cpu(), y, X.rounded(y, slack, "f16"), "out")
    graw = torch.zeros(T * K + 1, dtype=torch.float16, device=DEV)
    I8.expert_backward(outr[1:].view(T, N), cg, SCB.to(DEV), off, grad_X=graw[1:].view(T, K))
    g, slack = X.backward(outr[1:].view(T, N).cpu(), CB, SCB, off.cpu())
    X.check(graw[1:].view(T, K).cpu(), g, X.rounded(g, slack, "f16"), "grad_X")


def test_one_expert_is_the_projection(I8):
    """All rows in one segment: the projection's own forward and backward, to the rounding of its order of sums."""
    T, K, N = 300, 512, 384
    CB, SCB = gpu(*X.weights(1, N, K, 1))
    x, G = X.inputs(T, K, "bf16", 2).to(DEV), X.inputs(T, N, "bf16", 3, 0).to(DEV)
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    a, b = I8.expert_forward(x, CB, SCB, off), I8.int8_linear_forward(x, CB[0], SCB[0])
    y, slack = X.forward(x, CB, SCB, off)
    X.check(a, y, X.rounded(y, slack, "bf16"), "experts")
    X.check(b, y, X.rounded(y, slack, "bf16"), "projection")
    g, slack = X.backward(G, CB, SCB, off)
    X.check(I8.expert_backward(G, CB, SCB, off), g, X.rounded(g, slack, "bf16"), "experts' gradient")
    X.check(I8.int8_linear_backward_input(G, CB[0], SCB[0], False)[0], g, X.rounded(g, slack, "bf16"), "gradient")


def run_backward(I8, dt, R, N, K, off, ids=None, E=None, seed=1):
    E = len(off) - 1 if E is None else E
    CB, SCB = X.weights(E, N, K, seed)
    G = X.inputs(R, N, dt, seed + 1, 0)
    off = torch.tensor(off, dtype=torch.int32)
    ids = None if ids is None else torch.tensor(ids, dtype=torch.int32)
    G, CB, SCB, off, ids = gpu(G, CB, SCB, off, ids)
    got = I8.expert_backward(G, CB, SCB, off, ids)
    y, slack = X.backward(G, CB, SCB, off, ids)
    X.check(got, y, X.rounded(y, slack, dt), "grad_X")
    assert torch.equal(got, I8.expert_backward(G, CB, SCB, off, ids))
    return got


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,K", [(64, 64), (192, 128), (72, 200), (530, 1001), (8, 16), (1, 1), (1408, 136), (260, 24)])
def test_backward_sizes(I8, dt, N, K):
    run_backward(I8, dt, 45, N, K, [0, 0, 7, 40, 45])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("off", [[0, 1], [0, 129, 129, 256, 300], [0] * 40 + [3], [0, 15, 16, 17, 33, 64, 65],
                                 [0, 0, 0], [0, 255, 256, 700, 1200]])
def test_backward_segments(I8, dt, off):
    run_backward(I8, dt, max(off[-1], 1), 144, 160, off)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,E,N,K", [(1500, 2, 4, 264, 1100), (1500, 2, 4, 136, 4100), (800, 2, 3, 64, 3000),
                                       (2100, 3, 9, 400, 2304), (600, 1, 1, 8, 5000), (1500, 2, 4, 263, 1101),
                                       (800, 2, 3, 65, 3001), (700, 1, 2, 1001, 530), (700, 2, 3, 1, 259),
                                       (600, 1, 2, 40, 3), (520, 1, 1, 12, 1), (600, 1, 2, 100, 6)])
def test_backward_many_rows(I8, dt, T, k, E, N, K):
    off, _, _ = X.sort(X.choices(T, k, E, 7, 0.1, skew=1.5), E)
    run_backward(I8, dt, T * k, N, K, off.tolist())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,E,N,K", [(1500, 2, 4, 600, 1100), (900, 2, 3, 1041, 2101), (2100, 3, 9, 520, 2304),
                                       (600, 1, 1, 1028, 5000), (700, 2, 3, 577, 131), (64, 4, 64, 600, 1600),
                                       (64, 4, 64, 523, 1601), (40, 4, 70, 516, 1410)])
def test_backward_long_contractions(I8, dt, T, k, E, N, K):
    """Past what the tiles for short contractions take, with many rows an expert, and with few of them."""
    off, _, _ = X.sort(X.choices(T, k, E, 7, 0.1, skew=1.5), E)
    run_backward(I8, dt, T * k, N, K, off.tolist())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("width", [1101, 1102, 300, 2307])
def test_rows_off_borders(I8, dt, width):
    """Outputs whose rows start anywhere, from whole tiles, halves and quarters."""
    off, token, _ = X.sort(X.choices(1500, 2, 4, 7, 0.1, skew=1.5), 4)
    run_forward(I8, dt, 1500, 1040, width, off.tolist(), rows=token)
    run_backward(I8, dt, 3000, 600, width, off.tolist())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", [(2100, 1040, 900), (2100, 256, 1100), (60, 96, 80)])
@pytest.mark.parametrize("ids", [[-1, 0, -1, 1, 2, -1], [9, 9, 9, 9, 9, 2], [0, -1, -1, -1, -1, -1], [-1] * 6])
def test_segments_without_expert_among_others(I8, dt, T, K, N, ids):
    """Some of the experts are elsewhere: their rows are zeros, in every form, wherever they lie."""
    off = [0, T // 5, T // 5, T // 2, T // 2 + 3, T - 7, T - 2]
    got = run_forward(I8, dt, T, K, N, off, ids=ids, E=3)
    back = run_backward(I8, dt, T, N, K, off, ids=ids, E=3)
    for j, e in enumerate(ids):
        if not 0 <= e < 3:
            assert (got[off[j]:off[j + 1]] == 0).all() and (back[off[j]:off[j + 1]] == 0).all()
    assert (got[off[-1]:] == 0).all() and (back[off[-1]:] == 0).all()


def test_backward_rows_without_expert(I8):
    got = run_backward(I8, "bf16", 11, 80, 96, [0, 3, 6, 9], ids=[1, -1, 5], E=2)
    assert (got[3:] == 0).all() and (got[:3] != 0).any()


def test_backward_rows_without_expert_hide_nan(I8):
    """What lies in rows without an expert does not reach any row, NaN included."""
    CB, SCB = gpu(*X.weights(2, 64, 96, 1))
    G = X.inputs(50, 64, "f16", 2, 0).to(DEV)
    off = torch.tensor([0, 20, 30], dtype=torch.int32, device=DEV)
    a = I8.expert_backward(G, CB, SCB, off)
    G[30:] = float("nan")
    b = I8.expert_backward(G, CB, SCB, off)
    assert torch.equal(a, b) and (b[30:] == 0).all()


def test_backward_empty(I8):
    z = torch.zeros
    CB, SCB = z((2, 6, 8), dtype=torch.int8, device=DEV), z((2, 6), device=DEV)
    off = z(3, dtype=torch.int32, device=DEV)
    assert I8.expert_backward(z((0, 6), device=DEV), CB, SCB, off).shape == (0, 8)
    out = torch.full((4, 8), 7.0, device=DEV)
    I8.expert_backward(z((4, 0), device=DEV), CB[:, :0], SCB[:, :0], off + 4, grad_X=out)
    assert (out == 0).all()
    assert I8.expert_backward(z((4, 6), device=DEV), CB[:, :, :0], SCB, off).shape == (4, 0)


# ---- weighted sum ---------------------------------------------------------------------------------------------------


SUMS = [(1, 2, 8, 256), (33, 3, 5, 72), (50, 1, 4, 1), (64, 8, 16, 2048), (20, 64, 70, 40), (129, 2, 3, 4100),
        (3, 0, 2, 8), (0, 2, 2, 8), (17, 5, 9, 1023), (40, 4, 6, 513)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,E,N", SUMS)
@pytest.mark.parametrize("gated", [True, False])
def test_combine(I8, dt, T, k, E, N, gated):
    _, _, pos = X.sort(X.choices(T, k, E, 3, 0.2), E)
    g = torch.Generator().manual_seed(4)
    Y, base = (torch.randn(s, generator=g).to(TORCH[dt]) for s in ((T * k, N), (T, N)))
    gate = torch.rand((T, k), generator=g) if gated else None
    pos, Y, base, gate = gpu(pos, Y, base, gate)
    for b in (base, None):
        y, slack = X.combine(Y, pos, gate, b)
        got = I8.expert_combine(Y, pos, gate, b)
        X.check(got, y, X.rounded(y, slack, dt), "out")
    out = base.clone()
    assert I8.expert_combine(Y, pos, gate, out, out=out) is out
    assert torch.equal(out, I8.expert_combine(Y, pos, gate, base))


def test_combine_left_out_rows_and_repeats(I8):
    """Positions outside [0, R) are left out whatever their gate; a row may be named twice in the forward sum."""
    Y = torch.tensor([[1.0, 2.0], [float("inf"), 4.0], [5.0, float("nan")]], device=DEV)
    pos = torch.tensor([[0, 0], [-1, 2 ** 31 - 1], [3, 0]], dtype=torch.int32, device=DEV)
    gate = torch.tensor([[1.0, 2.0], [float("nan"), float("inf")], [float("inf"), 1.0]], device=DEV)
    assert I8.expert_combine(Y, pos, gate).tolist() == [[3.0, 6.0], [0.0, 0.0], [1.0, 2.0]]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,E,N", SUMS)
@pytest.mark.parametrize("gated", [True, False])
def test_combine_backward(I8, dt, T, k, E, N, gated):
    off, _, pos = X.sort(X.choices(T, k, E, 3, 0.2), E)
    g = torch.Generator().manual_seed(4)
    Y, G = (torch.randn(s, generator=g).to(TORCH[dt]) for s in ((T * k, N), (T, N)))
    gate = torch.rand((T, k), generator=g) if gated else None
    off, pos, Y, G, gate = gpu(off, pos, Y, G, gate)
    wY, wg, slack = X.combine_backward(G, pos, gate, Y, T * k)
    gY, gg = I8.expert_combine_backward(G, pos, gate, Y, n_rows=off[-1:])
    X.check(gY, wY, X.rounded(wY, 2.0 ** -24 * wY.abs(), dt), "grad_Y")
    X.check(gg, wg, X.rounded(wg, slack, "f32"), "grad_gate")
    only, none = I8.expert_combine_backward(G, pos, gate, n_rows=off[-1:], with_grad_gate=False)
    assert none is None and torch.equal(only, gY)
    none, only = I8.expert_combine_backward(G, pos, gate, Y, with_grad_Y=False)
    assert none is None and torch.equal(only, gg)


def test_combine_of_very_many_tokens(I8):
    """The most tokens there can be, and more workgroups than one axis of the grid is given."""
    for T, N in ((1 << 24, 1), ((1 << 20) + 3, 2048)):
        pos = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1).flip(0)
        Y = torch.arange(T, dtype=torch.float32, device=DEV)[:, None].repeat(1, N).bfloat16()
        want = Y.flip(0)
        assert torch.equal(I8.expert_combine(Y, pos), want)
        gY, gg = I8.expert_combine_backward(want, pos, None, Y, n_rows=pos[:1].view(1) + 1)
        assert torch.equal(gY, Y)
        assert torch.equal(gg, want[:, :1].float().square() * N)      # N equal terms, each exact: 16 bits squared


def test_combine_backward_leaves_unnamed_rows(I8):
    """Without n_rows, rows that no position names stay as they were; with it, those behind it become 0."""
    G = torch.ones((2, 16), device=DEV)
    pos = torch.tensor([[4, -1], [1, 9]], dtype=torch.int32, device=DEV)
    gY = torch.full((6, 16), 7.0, device=DEV)
    I8.expert_combine_backward(G, pos, None, with_grad_gate=False, rows=6, grad_Y=gY)
    assert gY[:, 0].tolist() == [7, 1, 7, 7, 1, 7]
    n = torch.tensor([5], dtype=torch.int32, device=DEV)
    I8.expert_combine_backward(G, pos, None, with_grad_gate=False, rows=6, grad_Y=gY, n_rows=n)
    assert gY[:, 0].tolist() == [7, 1, 7, 7, 1, 0]
    n.fill_(-3)                                                  # held inside [0, R]
    I8.expert_combine_backward(G, pos, None, with_grad_gate=False, rows=6, grad_Y=gY, n_rows=n + 100)
    assert gY[:, 0].tolist() == [7, 1, 7, 7, 1, 0]


# ---- together -------------------------------------------------------------------------------------------------------


def test_autograd_of_a_mixture(I8):
    """Sort, up projection, SiLU, down projection, weighted sum with a residual: gradients of the input and the gate
    against autograd over the dequantized weights in 64 bits, and the clipped AdamW step that follows."""
    T, k, E, K, H = 70, 2, 5, 96, 160
    torch.manual_seed(0)
    up, down = I8.Int8Experts(torch.randn(E, H, K, device=DEV) * K ** -0.5, threshold=0.0), \
        I8.Int8Experts(torch.randn(E, K, H, device=DEV) * H ** -0.5, threshold=0.0)
    ids = X.choices(T, k, E, 1, 0.1).to(DEV)
    x = torch.randn(T, K, device=DEV, requires_grad=True)
    gate = torch.rand(T, k, device=DEV, requires_grad=True)
    off, token, pos = I8.expert_sort(ids, E)
    h = up(x, off, rows=token, position=pos)
    y = I8.ExpertCombineFunction.apply(down(torch.nn.functional.silu(h), off), pos, gate, x, off[-1:])
    G = torch.randn_like(y)
    y.backward(G)

    xd, gd = x.detach().double().requires_grad_(), gate.detach().double().requires_grad_()
    Wu = torch.stack([X.dequantized(c, s) for c, s in zip(up.CB, up.SCB)])
    Wd = torch.stack([X.dequantized(c, s) for c, s in zip(down.CB, down.SCB)])
    z = xd.clone()
    for j in range(k):
        t = (ids[:, j] >= 0).nonzero()[:, 0]
        e = ids[t, j]
        hh = torch.nn.functional.silu((Wu[e] * xd[t][:, None]).sum(2))
        z = z.index_add(0, t, gd[t, j][:, None] * (Wd[e] * hh[:, None]).sum(2))
    z.backward(G.double())
    # 8-bit activations: a code is off by up to half of 1 / 127 of its row's largest, which is 3 to 4 of the row's rms:
    # at most 0.016 rms a value, 0.009 on average; two products in a row and the gate's sum add those as noise. The
    # gradient is taken at the quantized product's values (SiLU'), in fp16: the same size of error
    for got, want, what in ((y.detach(), z.detach(), "y"), (x.grad, xd.grad, "x"), (gate.grad, gd.grad, "gate")):
        err = float((got.double() - want).norm() / want.norm())
        assert err < 0.03, (what, err)

    p = [torch.nn.Parameter(x.detach().clone()), torch.nn.Parameter(gate.detach().clone())]
    p[0].grad, p[1].grad = x.grad.clone(), gate.grad.clone()
    opt = I8.AdamW(p, lr=0.1, weight_decay=0.0)
    norm, factor, bad = opt.grad_norm(1.0)
    opt.step(grad_scale=factor, found_inf=bad)
    want_norm, want_factor = X.grad_norm([x.grad, gate.grad], 1.0)
    assert abs(float(norm) - want_norm) <= 2.0 ** -23 * want_norm and float(bad) == 0
    assert abs(float(factor) - want_factor) <= 2.0 ** -23 * want_factor
    m = opt.state[p[0]]["m"]
    torch.testing.assert_close(m, 0.1 * x.grad * want_factor, rtol=1e-5, atol=0)


def test_autograd_refuses(I8):
    CB, SCB = gpu(*X.weights(2, 16, 32, 1))
    x = torch.randn(6, 32, device=DEV, requires_grad=True)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV)
    rows = torch.arange(6, dtype=torch.int32, device=DEV)
    y = I8.Int8ExpertsFunction.apply(x, CB, SCB, off, None, rows, None, 6.0)
    with pytest.raises(ValueError, match="position"):
        y.sum().backward()
    y = I8.Int8ExpertsFunction.apply(x, CB, SCB, off, None, None, None, 6.0)
    gx, = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()


def test_combine_function_without_n_rows(I8):
    """Rows that no position names get a gradient of 0."""
    Y = torch.randn(6, 8, device=DEV, requires_grad=True)
    pos = torch.tensor([[4, -1], [1, 9]], dtype=torch.int32, device=DEV)
    junk = torch.full((6, 8), float("nan"), device=DEV)
    del junk
    I8.ExpertCombineFunction.apply(Y, pos, None, None, None).sum().backward()
    assert Y.grad[:, 0].tolist() == [0, 1, 0, 0, 1, 0]


def test_replays_and_streams(I8):
    """Captured once, replayed with other inputs and eager work between: bit-identical to the eager calls. Two graphs
    and a side stream have workspaces of their own."""
    T, k, E, K, N = 90, 2, 4, 128, 96
    CB, SCB = gpu(*X.weights(E, N, K, 1))
    x, ids = X.inputs(T, K, "bf16", 2).to(DEV), X.choices(T, k, E, 1, 0.1).to(DEV)
    gate = torch.rand(T, k, device=DEV)

    def step(x, ids):
        off, token, pos = I8.expert_sort(ids, E)
        y = I8.expert_forward(x, CB, SCB, off, rows=token)
        out = I8.expert_combine(y, pos, gate)
        gY, gg = I8.expert_combine_backward(out, pos, gate, y, n_rows=off[-1:])
        gx = I8.expert_combine(I8.expert_backward(gY, CB, SCB, off), pos)
        return off, token, pos, y, out, gY, gg, gx, *I8.GradNormPlan([gx, gg]).norm(1.0)

    step(x, ids)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(x, ids)
        graphs.append((g, outs))
    side = torch.cuda.Stream()
    for i in range(4):
        x.copy_(X.inputs(T, K, "bf16", 20 + i).to(DEV))
        ids.copy_(X.choices(T, k, E, 30 + i, 0.2).to(DEV))
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        with torch.cuda.stream(side):
            there = step(x, ids)
        here = step(x, ids)
        torch.cuda.synchronize()
        for j, want in enumerate(here):
            assert torch.equal(there[j], want), ("stream", i, j)
            for _, outs in graphs:
                assert torch.equal(outs[j], want), ("replay", i, j)
