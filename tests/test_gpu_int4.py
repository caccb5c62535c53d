"""4-bit weights on the GPU: quantised and read back bit for bit, and the product
against float64.

Product tolerance.  The kernels sum x (16 + q) over a group, starting from
-(16 + z) times the group's fp32 sum of x, multiply by the scale and add the
groups up.  With g columns in a group and S = sum |x|: the sum of x is off by
g u S, times at most 31; the start's rounding by 31 u S; each of the g
additions by at most 2 u (truncating adders) of partial sums below 62 S.  So a
group is off by (31 g + 31 + 124 g) u S < 156 (g + 1) u S, times its scale;
adding the groups up, with the factor's rounding, by 2 (groups + 10) u of sum |x w| and as much of
the groups' own errors (left out, of second order, under the factor 1.01)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref_vocab as ref  # noqa: E402
from tests.ref_vocab import U  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32, dev, hidden  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu

KINDS = [(32, True, F32, F32, F32), (64, False, BF, BF, F32), (128, True, BF, BF, BF), (128, False, F32, F32, BF), (32, False, BF, BF, BF),
         (64, True, F32, BF, F32)]          # group, zeros, x, scales, y


def matrix(rng, rows, cols, group, zeros, sdtype):
    q = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    n, sld = ref.groups_of(cols, group), ref.scale_ld(cols, group)
    s = np.full((rows, sld), np.nan, np.float32)                # what lies past the groups does not count
    s[:, :n] = 2.0 ** rng.uniform(-8, -2, (rows, n))
    if sdtype == BF:
        s = ref.bf16(s)
    z = rng.integers(0, 256, (rows, sld)).astype(np.uint8)
    z[:, :n] = rng.integers(0, 16, (rows, n))
    codes = ref.pack(q, cols)
    z = z if zeros else None
    w = ng.Int4(dev(codes), dev(s, sdtype), rows, cols, group, None if z is None else dev(z))
    return w, ref.values4(codes, s, z, cols, group), s[:, :n].astype(np.float64)


def check(x, w, values, scales, group, ydtype):
    got = ng.ngram_project_int4(x, w, dtype=ydtype)
    xv = x.double().cpu().numpy()
    want = xv @ values.T
    k = xv.shape[1]
    n = scales.shape[1]
    size = np.zeros((xv.shape[0], n))
    for g in range(n):
        size[:, g] = np.abs(xv[:, g * group:(g + 1) * group]).sum(axis=1)
    bound = 1.01 * (156 * (min(group, k) + 1) * U * (size @ scales.T) + 2 * (n + 10) * U * (np.abs(xv) @ np.abs(values).T))
    bound += ref.half_step(np.abs(want) + bound, ydtype == BF)
    err = np.abs(got.double().cpu().numpy() - want)
    assert got.dtype == ydtype and got.shape == want.shape
    assert np.all(err <= bound), (err / bound).max()
    return got, err, want


SHAPES = [(1, 8, 1), (1, 2560, 2560), (2, 40, 300), (3, 136, 37), (16, 1032, 4103), (17, 264, 130), (31, 648, 16), (33, 128, 517), (64, 2568, 520),
          (65, 40, 7), (100, 1160, 33), (7, 4232, 70), (16, 6144, 17), (3, 6152, 40), (30, 3000, 40), (20, 8192, 264), (60, 1536, 100), (2, 16392, 9)]


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("n,k,o", SHAPES)
def test_product(n, k, o, kind):
    group, zeros, xt, st, yt = KINDS[kind]
    say(f"4-bit product {n} x {k} x {o} {KINDS[kind]}")
    rng = np.random.default_rng(n + 3 * k + 5 * o + kind)
    w, values, scales = matrix(rng, o, k, group, zeros, st)
    x = dev(hidden(rng, n, k).astype(np.float32), xt)
    got, err, want = check(x, w, values, scales, group, yt)
    if yt == F32 and k >= 128:
        # with rounding errors of random signs far below the bound
        assert np.linalg.norm(err) <= 4e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("n,k,o", [(1, 264, 33000), (5, 8, 33000), (20, 136, 32900), (40, 392, 33001), (70, 136, 32770), (4, 1032, 40001), (2, 6200, 33000),
                                   (40, 4104, 32801), (33, 2600, 32790), (9, 3208, 33333)])
def test_many_weight_rows(n, k, o):
    for kind in (0, 2, 5):
        group, zeros, xt, st, yt = KINDS[kind]
        say(f"4-bit product of many weight rows {n} x {k} x {o} {KINDS[kind]}")
        rng = np.random.default_rng(n + k + o + kind)
        w, values, scales = matrix(rng, o, k, group, zeros, st)
        check(dev(rng.normal(size=(n, k)).astype(np.float32), xt), w, values, scales, group, yt)


@pytest.mark.parametrize("n,o", [(3, 40), (40, 72), (3, 33000), (20, 33000), (64, 32800)])
def test_integers_are_exact(n, o):
    """Whole x and power-of-two scales: every partial sum is a whole number of units below 2^24."""
    say(f"4-bit integers n={n} o={o}")
    rng = np.random.default_rng(n)
    k, group = 1160, 64
    q, z = rng.integers(0, 16, (o, k)).astype(np.uint8), rng.integers(0, 16, (o, ref.scale_ld(k, group))).astype(np.uint8)
    s = 2.0 ** rng.integers(-2, 3, z.shape).astype(np.float32)
    for zeros in (True, False):
        w = ng.Int4(dev(ref.pack(q, k)), dev(s), o, k, group, dev(z) if zeros else None)
        x = rng.integers(-30, 31, (n, k)).astype(np.float32)
        want = x.astype(np.float64) @ ref.values4(ref.pack(q, k), s, z if zeros else None, k, group).T
        for xt in (BF, F32):
            got = ng.ngram_project_int4(dev(x, xt), w, dtype=F32)
            assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("o", [40, 33000])
def test_fp32_x_keeps_all_bits(o):
    """One column counts: y = x s (q - z), x with 24 significant bits, exact up to the last rounding and the 16's three bits."""
    say(f"fp32 x, o={o}")
    rng = np.random.default_rng(7)
    x = np.zeros((5, 64), np.float32)
    x[:, 9] = rng.normal(size=5)
    q = np.full((o, 64), 8, np.uint8)
    q[:, 9] = 15
    w = ng.Int4(dev(ref.pack(q, 64)), torch.ones(o, 4, device=DEV), o, 64, 32)
    got = ng.ngram_project_int4(dev(x), w, dtype=F32).double().cpu().numpy()
    want = 7.0 * x[:, 9:10].astype(np.float64)
    # x 31 in three parts, less 24 x: four roundings of at most 31 |x| u, doubled
    assert np.all(np.abs(got - want) <= 8 * 31 / 7 * U * np.abs(want))


@pytest.mark.parametrize("o", [40, 33000])
@pytest.mark.parametrize("n", [3, 20, 64])
def test_a_row_s_nan_stays_in_it(n, o):
    say(f"4-bit NaN n={n} o={o}")
    rng = np.random.default_rng(n)
    w, values, scales = matrix(rng, o, 264, 64, True, F32)
    for xt in (BF, F32):
        x = rng.normal(size=(n, 264)).astype(np.float32)
        clean = ng.ngram_project_int4(dev(x, xt), w, dtype=F32)
        x[1, 200], x[2, 7] = np.nan, np.inf
        got = ng.ngram_project_int4(dev(x, xt), w, dtype=F32)
        assert torch.all(torch.isnan(got[1])) and not torch.any(torch.isfinite(got[2]))
        keep = [i for i in range(n) if i not in (1, 2)]
        assert torch.equal(got[keep], clean[keep])


def test_nothing_past_the_result_and_no_rows():
    say("4-bit guard bytes")
    rng = np.random.default_rng(1)
    for o in (37, 33001):
        w, values, scales = matrix(rng, o, 136, 32, True, BF)
        for n in (1, 17, 66):
            x = torch.randn(n, 136, device=DEV)
            for dtype in (BF, F32):
                wide = torch.full(((n + 2) * o,), float("nan"), dtype=dtype, device=DEV)
                ng.ngram_project_int4(x, w, out=wide)
                assert torch.all(torch.isnan(wide[n * o:])) and torch.all(torch.isfinite(wide[:n * o]))
        assert ng.ngram_project_int4(torch.empty(0, 136, device=DEV), w).shape == (0, o)
    empty = ng.Int4.empty(0, 136)
    assert ng.ngram_project_int4(torch.randn(3, 136, device=DEV), empty).shape == (3, 0)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 40), (5, 136), (200, 264), (33, 2560), (7, 1032), (1000, 64), (2, 8192)])
def test_quantise_and_read_back(rows, cols, group):
    say(f"4-bit quantise {rows} x {cols} group {group}")
    rng = np.random.default_rng(rows + cols + group)
    base = (rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1)))).astype(np.float32)
    base[0, :8] = 0.0
    for xt in (F32, BF):
        x = base if xt == F32 else ref.bf16(base)
        for asym in (True, False):
            for st in (F32, BF):
                got = ng.ngram_quant_int4(dev(x, xt), group, zeros=asym, scale_dtype=st)
                q, s, z = ref.quant4(x, group, asym, st == BF)
                n = ref.groups_of(cols, group)
                assert np.array_equal(ref.unpack(got.codes.cpu().numpy(), cols), q)
                assert np.array_equal(got.scales.float().cpu().numpy()[:, :n], s) and torch.all(got.scales[:, n:] == 1)
                assert (got.zeros is None) == (not asym)
                if asym:
                    assert np.array_equal(got.zeros.cpu().numpy()[:, :n], z) and torch.all(got.zeros[:, n:] == 8)
                value = ref.values4(ref.pack(q, cols), s, z, cols, group)
                back = ng.ngram_dequant_int4(got)
                assert np.array_equal(back.cpu().numpy(), value.astype(np.float32))
                assert torch.equal(ng.ngram_dequant_int4(got, dtype=BF), back.to(BF))


def test_quantise_strange_values():
    say("4-bit strange values")
    x = np.random.default_rng(3).normal(size=(9, 128)).astype(np.float32)
    x[0, 3], x[1, 70], x[2, 0], x[3] = np.nan, np.inf, -np.inf, 0.0
    x[4, :32], x[5, 5] = np.abs(x[4, :32]) + 1, 3e38
    x[5, 6], x[6, :64], x[7, :32] = -3e38, 1e-40, -1e-45
    x[8, 64:] = -0.0
    for asym in (True, False):
        for st in (F32, BF):
            got = ng.ngram_quant_int4(dev(x), 32, zeros=asym, scale_dtype=st)
            q, s, z = ref.quant4(x, 32, asym, st == BF)
            assert np.array_equal(ref.unpack(got.codes.cpu().numpy(), 128), q)
            assert np.array_equal(got.scales.float().cpu().numpy()[:, :4], s, equal_nan=True)
            if asym:
                assert np.array_equal(got.zeros.cpu().numpy()[:, :4], z)
            nan = np.isnan(ng.ngram_dequant_int4(got).cpu().numpy()).reshape(9, 4, 32)
            assert np.array_equal(nan.all(axis=2), np.isnan(s)) and np.array_equal(nan.any(axis=2), np.isnan(s))
            assert nan[0, 0].all() and nan[1, 2].all() and nan[2, 0].all() and not nan[3].any()


def test_reused_buffers_and_a_given_stream():
    say("4-bit out= and stream=")
    x = torch.randn(33, 264, device=DEV)
    plain = ng.ngram_quant_int4(x, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = ng.Int4.empty(33, 264, 64, zeros=True, stream=side)
    ng.ngram_quant_int4(x, out=again, stream=side)
    y = ng.ngram_project_int4(x, again, dtype=F32, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again.codes, plain.codes) and torch.equal(again.zeros, plain.zeros)
    assert torch.equal(y, ng.ngram_project_int4(x, plain, dtype=F32))


def test_quotients_are_those_of_a_division():
    """33 million fp32 weights in groups of every spread, and bf16 ones, whose quotients lie on halves often: the codes that
    correctly rounded divisions give."""
    say("4-bit quotients")
    g = torch.Generator(device=DEV).manual_seed(1)
    for dtype in (F32, BF):
        x = (torch.randn((4096, 8192), generator=g, device=DEV) * torch.exp2(torch.randint(-90, 90, (4096, 1), generator=g, device=DEV).float())).to(dtype)
        for st in (F32, BF):
            got = ng.ngram_quant_int4(x, 32, zeros=True, scale_dtype=st)
            s, z = got.scales.float()[:, :, None], got.zeros.float()[:, :, None]
            want = (torch.round(x.float().view(4096, 256, 32) / s) + z).clamp(0, 15).to(torch.uint8).view(4096, -1)
            codes = torch.stack((got.codes & 15, got.codes >> 4), dim=2).view(4096, -1)
            assert torch.equal(codes, want)
