"""ngram_project_fp8 on the GPU against the float64 product of the decoded
operands.

Tolerances.  An fp32 result sums exact bf16 products in fp32: within
(K + 8) u of the sum of absolute terms (any order), doubled for truncating
adders.  A bf16 result comes from the 8-bit matrix instruction, which keeps
at least 10 bits below the largest product of each block of 128, and is rounded to bf16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref8  # noqa: E402
from tests.ref8 import U  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32, dev, hidden  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu


def fp8(codes, scales, cols, tile=False):
    return ng.Fp8(dev(codes), dev(scales), codes.shape[0], cols, block_rows=128 if tile else 1)


def operands(rng, m, n, k, tile):
    a, b = ref8.quant(hidden(rng, m, k)), ref8.quant(rng.normal(size=(n, k)) * np.exp(rng.normal(size=(n, 1))), tile)
    return a, b


def check(m, n, k, a, b, tile, dtype, a_tile=False):
    av, bv = ref8.values(*a, k, tile=a_tile), ref8.values(*b, k, tile=tile)
    want = av @ bv.T
    size = np.abs(av) @ np.abs(bv).T
    got = ng.ngram_project_fp8(fp8(*a, k, a_tile), fp8(*b, k, tile), dtype=dtype)
    assert got.shape == (m, n) and got.dtype == dtype
    err = np.abs(got.double().cpu().numpy() - want)
    if dtype == F32:
        assert np.all(err <= 2 * (k + 8) * U * size)
        assert np.linalg.norm(err) <= 1e-6 * np.linalg.norm(want)
    else:
        worst = np.zeros_like(want)
        for at in range(0, k, 128):
            worst += (np.abs(av[:, None, at:at + 128]).max(axis=2) * np.abs(bv[:, at:at + 128]).max(axis=1)[None]) * 2.0 ** -9
        assert np.all(err <= ref8.bf16_half_step(want) * (1 + 2.0 ** -6) + worst + 2 * (k + 8) * U * size)
        assert np.linalg.norm(err) <= 3e-3 * np.linalg.norm(want)
    return got


SHAPES = [(1, 8, 8), (1, 2560, 2560), (4, 264, 136), (16, 128, 1024), (17, 40, 392), (33, 256, 128), (64, 1032, 520), (65, 8, 8),
          (65, 1032, 520), (128, 128, 128), (200, 264, 2568), (777, 520, 264), (1024, 2560, 640), (300, 136, 4232), (4100, 4104, 136)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, dtype):
    for tile in (True, False):
        say(f"product {m} x {n} x {k} {dtype} tile={tile}")
        a, b = operands(np.random.default_rng(m + 3 * n + 5 * k), m, n, k, tile)
        check(m, n, k, a, b, tile, dtype)


@pytest.mark.parametrize("m,n,k", [(7900, 2552, 136), (8192, 2560, 100), (4090, 5000, 1032), (16300, 2552, 640), (2500, 7672, 1544)])
def test_many_rows_and_columns(m, n, k):
    """Results that fill the card's rounds with the largest tiles, with ragged edges; one, few and many steps of K."""
    say(f"large product {m} x {n} x {k}")
    a, b = operands(np.random.default_rng(m + n + k), m, n, k, False)
    check(m, n, k, a, b, False, BF)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", [(136, 264, 16392), (264, 520, 5000), (520, 264, 4097), (72, 8, 8200)])
def test_long_k_is_split(m, n, k, dtype):
    """Weight-gradient shapes: K is the tokens, both operands scaled along them."""
    say(f"long K {m} x {n} x {k} {dtype}")
    rng = np.random.default_rng(k)
    a, b = ref8.quant(rng.normal(size=(m, k)) * np.exp(rng.normal(size=(m, 1)))), ref8.quant(rng.normal(size=(n, k)))
    check(m, n, k, a, b, False, dtype)


def test_both_operands_tiled():
    say("both operands with tile scales")
    rng = np.random.default_rng(2)
    m, n, k = 300, 264, 392
    a, b = ref8.quant(hidden(rng, m, k), tile=True), ref8.quant(hidden(rng, n, k), tile=True)
    check(m, n, k, a, b, True, F32, a_tile=True)
    check(m, n, k, a, b, True, BF, a_tile=True)


@pytest.mark.parametrize("m", [3, 100, 600])
def test_integers_are_exact(m):
    """Small integers with power-of-two scales: every partial sum is a multiple of one unit below 2^24 of it."""
    say(f"integers m={m}")
    rng = np.random.default_rng(m)
    n, k = 264, 1160
    codes = lambda r: (ref8.code_of(rng.integers(0, 9, (r, ref8.code_shape(r, k)[1])).astype(float))  # noqa: E731
                       | (rng.integers(0, 2, (r, ref8.code_shape(r, k)[1])) << 7)).astype(np.uint8)
    a, b = codes(m), codes(n)
    a[:, k:] = b[:, k:] = 0
    sa = rng.integers(124, 131, (m, ref8.scale_cols(k))).astype(np.uint8)
    sb = rng.integers(124, 131, (n, ref8.scale_cols(k))).astype(np.uint8)
    want = ref8.values(a, sa, k) @ ref8.values(b, sb, k).T
    got = ng.ngram_project_fp8(fp8(a, sa, k), fp8(b, sb, k), dtype=F32)
    assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("m,dtype", [(5, F32), (100, F32), (100, BF), (600, BF)])
def test_nan_stays_in_its_row_and_column(m, dtype):
    say(f"NaN m={m} {dtype}")
    rng = np.random.default_rng(m)
    n, k = 136, 264
    (ac, asc), (bc, bsc) = operands(rng, m, n, k, False)
    ac[2, 200] = 0x7F
    bc[7, 0] = 0xFF
    got = ng.ngram_project_fp8(fp8(ac, asc, k), fp8(bc, bsc, k), dtype=dtype).float().cpu().numpy()
    nan = np.zeros((m, n), bool)
    nan[2], nan[:, 7] = True, True
    assert np.array_equal(np.isnan(got), nan)


def test_no_rows_and_nothing_past_the_result():
    say("no rows; guard bytes")
    b = ng.ngram_quant_fp8(torch.randn(64, 128, device=DEV))[0]
    assert ng.ngram_project_fp8(ng.Fp8.empty(0, 128), b).shape == (0, 64)
    for m in (1, 37, 130):
        a = ng.ngram_quant_fp8(torch.randn(m, 128, device=DEV))[0]
        for dtype in (BF, F32):
            wide = torch.full(((m + 4) * 64,), float("nan"), dtype=dtype, device=DEV)
            ng.ngram_project_fp8(a, b, out=wide)
            assert torch.all(torch.isnan(wide[m * 64:])) and torch.all(torch.isfinite(wide[:m * 64]))


def test_layer_gradients_end_to_end():
    """y = P x with both gradients through the quantisers, against the same in float64 on the quantised values."""
    say("layer and its gradients")
    rng = np.random.default_rng(11)
    n, d_in, d_out = 392, 264, 520
    x, P, dy = (torch.from_numpy(v).to(DEV) for v in (hidden(rng, n, d_in), rng.normal(size=(d_out, d_in)), rng.normal(size=(n, d_out))))
    x, P, dy = x.to(BF), P.float(), dy.to(BF)
    xq, xt = ng.ngram_quant_fp8(x, transposed=True)
    Pq, Pt = ng.ngram_quant_fp8(P, transposed=True, block_rows=128)
    gq, gt = ng.ngram_quant_fp8(dy, transposed=True)
    val = lambda q: ref8.values(q.codes.view(torch.uint8).cpu().numpy(), q.scales.cpu().numpy(), q.cols, q.block_rows == 128)  # noqa: E731
    for a, b in ((xq, Pq), (gq, Pt), (gt, xt)):
        got = ng.ngram_project_fp8(a, b, dtype=F32).double().cpu().numpy()
        want = val(a) @ val(b).T
        assert np.linalg.norm(got - want) <= 1e-6 * np.linalg.norm(want)
    assert np.array_equal(val(Pq).T, val(Pt))


def test_other_stream_and_graph():
    say("stream and graph")
    rng = np.random.default_rng(9)
    sets = [(4, 2560, 2560), (300, 264, 264), (136, 264, 16392), (600, 2560, 2560)]
    calls = []
    for m, n, k in sets:
        a, b = (ng.ngram_quant_fp8(dev(rng.normal(size=(r, k)), F32))[0] for r in (m, n))
        calls.append((a, b, torch.empty((m, n), dtype=F32, device=DEV), ng.project_fp8_workspace(m, n, k)))
    assert any(c[3] is not None for c in calls)

    def work():
        for a, b, out, ws in calls:
            ng.ngram_project_fp8(a, b, out=out, workspace=ws)

    work()
    torch.cuda.synchronize()
    want = [c[2].clone() for c in calls]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        work()
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            work()
    for _ in range(4):
        for c in calls:
            c[2].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(c[2], w) for c, w in zip(calls, want))


def test_refusals():
    say("refusals of the binding")
    a, b = ng.ngram_quant_fp8(torch.randn(4, 64, device=DEV))[0], ng.ngram_quant_fp8(torch.randn(16, 64, device=DEV))[0]
    other = ng.ngram_quant_fp8(torch.randn(16, 128, device=DEV))[0]
    nine = ng.ngram_quant_fp8(torch.randn(9, 64, device=DEV))[0]
    long = [ng.ngram_quant_fp8(torch.randn(136, 16392, device=DEV))[0] for _ in range(2)]
    bad = [
        lambda: ng.ngram_project_fp8(a, other),
        lambda: ng.ngram_project_fp8(a, nine),
        lambda: ng.ngram_project_fp8(a, b, dtype=torch.float16),
        lambda: ng.ngram_project_fp8(a, b, out=torch.empty(4, 15, device=DEV)),
        lambda: ng.ngram_project_fp8(*long, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
        lambda: ng.project_fp8_workspace(4, 12, 64),
        lambda: ng.project_fp8_workspace(4, 16, (1 << 23) + 1),
    ]
    for f in bad:
        with pytest.raises(ng.NgramError):
            f()
