"""ngram_quant_fp8, ngram_add_norm and ngram_add_norm_grad on the GPU against
the float64 forms of tests/ref8.py.

Tolerances.  Quantisation scales by a power of two and rounds once: bytes are
equal.  The norm's sum is an fp32 add and a bf16 rounding: bits are equal.  r
comes from a sum of d positive fp32 terms added over at most 8 + 128 / 16 + 6
+ 16 steps, halved by the root, plus four operations: within 32 u.  A value
y = s r gamma then lies within 35 u of its float64 form before its last
rounding, which may go either way where a midpoint lies that near."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref8  # noqa: E402
from tests.ref8 import U  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def host(t):
    return (t.float() if t.dtype == BF else t).cpu().numpy()


def rounded(x, dtype):
    x = np.asarray(x, dtype=np.float32)
    return ref8.bf16(x) if dtype == BF else x


def hidden(rng, n, d):
    """Rows with a few large columns."""
    return rng.normal(size=(n, d)) * np.exp(0.5 * rng.normal(size=d)) * np.where(rng.random(d) < 0.02, 30, 1)


def same_codes(got, want):
    got, want = got.view(torch.uint8).cpu().numpy(), want
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal((got & 0x7F) == 0x7F, nan)
    assert np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,d", [(1, 8), (3, 136), (128, 128), (129, 1032), (300, 520), (517, 256), (640, 8)])
def test_quant_bytes(n, d, dtype):
    say(f"quant n={n} d={d} {dtype}")
    rng = np.random.default_rng(n * 1000 + d)
    x = rounded(hidden(rng, n, d) * 10.0 ** rng.integers(-6, 6, (n, 1)), dtype)
    if n > 100:
        x[5:9] = 0.0                                    # blocks of zeros
        x[n // 2, :] *= np.float32(2.0 ** -120)         # below the smallest scale
    x = rounded(x, dtype)                               # the numbers that the call is given
    q, qt = ng.ngram_quant_fp8(dev(x, dtype), rows=True, transposed=True)
    for got, want in ((q, ref8.quant(x.astype(np.float64))), (qt, ref8.quant(x.T.astype(np.float64)))):
        same_codes(got.codes, want[0])
        assert np.array_equal(got.scales.cpu().numpy(), want[1])
    alone, none = ng.ngram_quant_fp8(dev(x, dtype))
    assert none is None and torch.equal(alone.codes.view(torch.uint8), q.codes.view(torch.uint8))
    w, wt = ng.ngram_quant_fp8(dev(x, dtype), transposed=True, block_rows=128)
    for got, want in ((w, ref8.quant(x.astype(np.float64), tile=True)), (wt, ref8.quant(x.T.astype(np.float64), tile=True))):
        same_codes(got.codes, want[0])
        assert np.array_equal(got.scales.cpu().numpy(), want[1])


def test_quant_not_finite():
    say("quant of infinities and NaN")
    rng = np.random.default_rng(7)
    x = rng.normal(size=(200, 264)).astype(np.float32)
    x[0, 3], x[1, 140], x[150, 263], x[199, 0] = np.inf, -np.inf, np.nan, np.nan
    x[60] = np.nan                                      # a row of nothing else
    for tile in (False, True):
        q, qt = ng.ngram_quant_fp8(dev(x), transposed=True, block_rows=128 if tile else 1)
        for got, want in ((q, ref8.quant(x.astype(np.float64), tile)), (qt, ref8.quant(x.T.astype(np.float64), tile))):
            same_codes(got.codes, want[0])
            assert np.array_equal(got.scales.cpu().numpy(), want[1])


NORM_SHAPES = [(1, 8), (1, 2560), (4, 2560), (5, 520), (77, 1032), (300, 8192), (2048, 2560), (2050, 136), (2049, 4104),
               (2100, 1536), (3, 16392), (2, 65536), (2048, 8200)]


@pytest.mark.parametrize("n,d", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_add_norm(n, d, dtype):
    say(f"add_norm n={n} d={d} {dtype}")
    rng = np.random.default_rng(n + 7 * d)
    x, res = rounded(rng.normal(size=(n, d)) * 0.1, dtype), rounded(hidden(rng, n, d), BF)
    gamma = (1 + 0.2 * rng.normal(size=d)).astype(np.float32)
    res[n // 2] = -x[n // 2] if dtype == BF else 0      # a row that is (nearly) zero
    total = torch.empty((n, d), dtype=BF, device=DEV)
    out = ng.ngram_add_norm(dev(x, dtype), dev(gamma), EPS, residual=dev(res, BF), sum_out=total, keep_y=True, keep_r=True)
    s, r, y = ref8.add_norm(x, res, gamma, EPS)
    assert np.array_equal(host(total), s.astype(np.float32))
    assert np.all(np.abs(host(out.r) - r) <= 32 * U * r)
    near = 35 * U * np.abs(y)
    assert np.all(np.abs(host(out.y) - y) <= ref8.bf16_half_step(y) * (1 + 2.0 ** -7) + near)
    check_codes(out.q, y, 35 * U)
    # each output alone, the residual updated in place, and no residual
    again = dev(res, BF)
    ng.ngram_add_norm(dev(x, dtype), dev(gamma), EPS, residual=again, sum_out=again, quantise=False)
    assert torch.equal(again, total)
    lone = ng.ngram_add_norm(total, dev(gamma), EPS)
    assert lone.sum is None and lone.y is None and torch.equal(lone.q.codes.view(torch.uint8), out.q.codes.view(torch.uint8))
    assert torch.equal(lone.q.scales, out.q.scales)


def check_codes(q, y, rel):
    """Codes and scales of y known to `rel`: equal up to roundings that can go either way."""
    n, d = y.shape
    codes, scales = q.codes.view(torch.uint8).cpu().numpy(), q.scales.cpu().numpy()
    nb = ref8.ceil_div(d, 128)
    am = ref8.block_max(ref8.padded(y))
    lo, hi = ref8.exponent(am * (1 - rel)), ref8.exponent(am * (1 + rel))
    e = scales[:, :nb].astype(int) - 127
    assert np.all((e == lo) | (e == hi))
    assert np.all(scales[:, nb:] == 127) and np.all(codes[:, d:] == 0)
    got = ref8.values(codes, scales, d)
    scale = np.repeat(2.0 ** e, 128, axis=1)[:, :d]
    # near a power of two the spacing is that of the larger side
    half = ref8.step_at(np.abs(y) * (1 + rel) / scale) / 2 * scale
    assert np.all(np.abs(got - y) <= half + rel * np.abs(y))


def test_add_norm_rows_that_overflow_or_are_not_finite():
    say("add_norm with infinities, NaN, overflow and zeros")
    n, d = 6, 1032
    rng = np.random.default_rng(3)
    x = rounded(rng.normal(size=(n, d)), BF)
    x[1, 5], x[2, 700], x[3] = np.inf, np.nan, 0.0
    x[4] = rounded(np.full(d, 3e38), BF)                # the sum of squares overflows: r = 0
    gamma = np.ones(d, dtype=np.float32)
    out = ng.ngram_add_norm(dev(x, BF), dev(gamma), 0.0, keep_y=True, keep_r=True)
    good = [0, 5]
    _, r, y = ref8.add_norm(x, np.zeros((n, d), np.float32), gamma, 0.0)
    assert np.all(np.abs(host(out.y)[good] - y[good]) <= ref8.bf16_half_step(y[good]) * 1.01 + 35 * U * np.abs(y[good]))
    h = host(out.y)
    assert np.isnan(h[1, 5]) and np.all(h[1, :5] == 0) and np.all(np.isnan(h[2])) and np.all(np.isnan(h[3]))
    assert np.all(h[4] == 0) and host(out.r)[4] == 0
    codes = out.q.codes.view(torch.uint8).cpu().numpy()
    assert np.all((codes[3, :d] & 0x7F) == 0x7F) and np.all(codes[:, d:] == 0) and np.all(codes[4] == 0)
    zero = ng.ngram_add_norm(dev(x[3:4], BF), dev(gamma), 1e-6, keep_y=True)
    assert torch.all(zero.y == 0) and torch.all(zero.q.codes.view(torch.uint8) == 0) and torch.all(zero.q.scales == 127)


GRAD_SHAPES = [(1, 8), (1, 2560), (4, 2560), (777, 520), (300, 1032), (2048, 2560), (5000, 136), (2049, 4104), (2, 65536),
               (2048, 8200), (2500, 16392)]


@pytest.mark.parametrize("n,d", GRAD_SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_add_norm_grad(n, d, dtype):
    say(f"add_norm_grad n={n} d={d} {dtype}")
    rng = np.random.default_rng(n + 11 * d)
    s, dsum = rounded(hidden(rng, n, d), BF), rounded(rng.normal(size=(n, d)) * 0.01, BF)
    dy = rounded(rng.normal(size=(n, d)) * 0.01, dtype)
    gamma = (1 + 0.2 * rng.normal(size=d)).astype(np.float32)
    r = (1 / np.sqrt((s.astype(np.float64) ** 2).mean(axis=1) + EPS)).astype(np.float32)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    want, want_g, size, size_g = ref8.add_norm_grad(f(dy), f(s), f(r), f(gamma), f(dsum))
    dx, dg = ng.ngram_add_norm_grad(dev(dy, dtype), dev(s, BF), dev(r), dev(gamma), dsum=dev(dsum, BF))
    # the row's sum: at most 8 + 8 + 6 + 16 additions and three roundings a term; then six operations
    assert np.all(np.abs(host(dx) - want) <= ref8.bf16_half_step(want) * (1 + 2.0 ** -7) + 50 * U * size)
    # a column's sum: the rows of one wavefront, then at most 512 partial sums
    assert np.all(np.abs(host(dg) - want_g) <= (ref8.ceil_div(n, 512) + 540) * U * size_g)
    plain, _ = ng.ngram_add_norm_grad(dev(dy, dtype), dev(s, BF), dev(r), dev(gamma))
    zero, _ = ng.ngram_add_norm_grad(dev(dy, dtype), dev(s, BF), dev(r), dev(gamma), dsum=torch.zeros_like(dx))
    assert torch.equal(plain, zero)
    over = dev(dsum, BF)                                # dx in the place of dsum
    again, dg2 = ng.ngram_add_norm_grad(dev(dy, dtype), dev(s, BF), dev(r), dev(gamma), dsum=over, dx_out=over)
    assert torch.equal(again, dx) and torch.equal(dg2, dg)
    if dtype == BF:                                     # and in the place of dy
        own = dev(dy, BF)
        again, _ = ng.ngram_add_norm_grad(own, dev(s, BF), dev(r), dev(gamma), dsum=dev(dsum, BF), dx_out=own)
        assert torch.equal(again, dx)


@pytest.mark.parametrize("n,d", [(5, 24), (127, 40), (513, 2560), (1024, 8), (1024, 4096), (1025, 40), (513, 8192), (900, 1032)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_add_norm_grad_at_the_edge_of_few_rows(n, d, dtype):
    """Up to 1024 rows and 2^22 elements one launch computes both gradients, unless dx takes dy's place."""
    say(f"add_norm_grad, few rows n={n} d={d} {dtype}")
    rng = np.random.default_rng(3 * n + d)
    s, dy = rounded(hidden(rng, n, d), BF), rounded(rng.normal(size=(n, d)) * 0.01, dtype)
    gamma = (1 + 0.2 * rng.normal(size=d)).astype(np.float32)
    r = (1 / np.sqrt((s.astype(np.float64) ** 2).mean(axis=1) + EPS)).astype(np.float32)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    want, want_g, size, size_g = ref8.add_norm_grad(f(dy), f(s), f(r), f(gamma), np.zeros((n, d)))
    dx, dg = ng.ngram_add_norm_grad(dev(dy, dtype), dev(s, BF), dev(r), dev(gamma))
    assert np.all(np.abs(host(dx) - want) <= ref8.bf16_half_step(want) * (1 + 2.0 ** -7) + 50 * U * size)
    # a column's sum: every 128th row by one thread, joins of 4 and 32, two roundings a term; with two launches up to 512 partial sums
    assert np.all(np.abs(host(dg) - want_g) <= 560 * U * size_g)
    if dtype == BF:
        own = dev(dy, BF)
        again, dg2 = ng.ngram_add_norm_grad(own, dev(s, BF), dev(r), dev(gamma), dx_out=own)
        assert torch.equal(again, dx)
        assert np.all(np.abs(host(dg2) - want_g) <= 560 * U * size_g)


@pytest.mark.parametrize("n,d", [(20001, 8), (9001, 136), (6024, 520), (5003, 1032), (2049, 1544), (1030, 2048), (1100, 1000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_add_norm_grad_of_many_narrow_rows(n, d, dtype):
    """A workgroup takes several narrow rows at once, the last of them past the end."""
    say(f"add_norm_grad, narrow rows n={n} d={d} {dtype}")
    rng = np.random.default_rng(5 * n + d)
    s, dsum = rounded(hidden(rng, n, d), BF), rounded(rng.normal(size=(n, d)) * 0.01, BF)
    dy = rounded(rng.normal(size=(n, d)) * 0.01, dtype)
    gamma = (1 + 0.2 * rng.normal(size=d)).astype(np.float32)
    r = (1 / np.sqrt((s.astype(np.float64) ** 2).mean(axis=1) + EPS)).astype(np.float32)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    want, want_g, size, size_g = ref8.add_norm_grad(f(dy), f(s), f(r), f(gamma), f(dsum))
    dx, dg = ng.ngram_add_norm_grad(dev(dy, dtype), dev(s, BF), dev(r), dev(gamma), dsum=dev(dsum, BF))
    assert np.all(np.abs(host(dx) - want) <= ref8.bf16_half_step(want) * (1 + 2.0 ** -7) + 50 * U * size)
    # a column's sum: the rows of one wavefront, up to 16 slots, then at most 512 partial sums
    assert np.all(np.abs(host(dg) - want_g) <= (ref8.ceil_div(n, 512) + 556) * U * size_g)


def test_no_rows():
    say("no rows")
    d = 264
    g = torch.ones(d, device=DEV)
    e = lambda dt=BF: torch.empty((0, d), dtype=dt, device=DEV)  # noqa: E731
    out = ng.ngram_add_norm(e(), g, EPS, keep_y=True, keep_r=True)
    assert out.y.shape == (0, d) and out.q.rows == 0
    dx, dg = ng.ngram_add_norm_grad(e(), e(), torch.empty(0, device=DEV), g, dgamma_out=torch.full((d,), 7.0, device=DEV))
    assert dx.shape == (0, d) and torch.all(dg == 0)
    q, _ = ng.ngram_quant_fp8(e(F32))
    assert q.rows == 0
    torch.cuda.synchronize()


def test_norm_gradient_against_differences():
    """dL/dx of the whole GPU forward and backward against central differences of the float64 forward, L = sum(w y)."""
    say("gradient against differences")
    rng = np.random.default_rng(5)
    n, d, t = 4, 136, 1e-4
    s, w = rounded(rng.normal(size=(n, d)), BF), rounded(rng.normal(size=(n, d)), BF)
    gamma = (1 + 0.2 * rng.normal(size=d)).astype(np.float32)
    fwd = ng.ngram_add_norm(dev(s, BF), dev(gamma), EPS, sum_out=torch.empty((n, d), dtype=BF, device=DEV), quantise=False, keep_r=True)
    dx, dg = ng.ngram_add_norm_grad(dev(w, BF), fwd.sum, fwd.r, dev(gamma))

    def loss(s, gamma):
        return (s / np.sqrt((s * s).mean(axis=1, keepdims=True) + EPS) * gamma * w).sum()

    s64, g64 = s.astype(np.float64), gamma.astype(np.float64)
    for i, j in zip(rng.integers(0, n, 40), rng.integers(0, d, 40)):
        e = np.zeros((n, d))
        e[i, j] = t
        diff = (loss(s64 + e, g64) - loss(s64 - e, g64)) / (2 * t)
        # central differences of a function with third derivatives of order 10: t^2 * 10; dx is a bf16 value
        assert abs(host(dx)[i, j] - diff) <= 10 * t * t + 2.0 ** -8 * abs(diff) + 1e-5
        e = np.zeros(d)
        e[j] = t
        assert abs(host(dg)[j] - (loss(s64, g64 + e) - loss(s64, g64 - e)) / (2 * t)) <= 1e-4


def test_other_stream_and_graph():
    """A side stream, and graph replays with eager work between them, give the eager bits."""
    say("stream and graph")
    n, d = 700, 2560
    rng = np.random.default_rng(9)
    x, res, gamma = dev(rng.normal(size=(n, d)), BF), dev(rng.normal(size=(n, d)), BF), dev(np.ones(d, np.float32))
    total, y, r = torch.empty((n, d), dtype=BF, device=DEV), torch.empty((n, d), dtype=BF, device=DEV), torch.empty(n, device=DEV)
    q, dx, dg = ng.Fp8.empty(n, d), torch.empty((n, d), dtype=BF, device=DEV), torch.empty(d, device=DEV)
    qt, ws = ng.Fp8.empty(d, n), ng.add_norm_grad_workspace(n, d)

    def work():
        ng.ngram_add_norm(x, gamma, EPS, residual=res, sum_out=total, y_out=y, q_out=q, r_out=r)
        ng.ngram_add_norm_grad(y, total, r, gamma, dsum=res, dx_out=dx, dgamma_out=dg, workspace=ws)
        ng.ngram_quant_fp8(dx, rows=False, qt=qt)

    outs = (total, y, r, q.codes.view(torch.uint8), q.scales, dx, dg, qt.codes.view(torch.uint8), qt.scales)
    work()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        for o in outs:
            o.zero_()
        work()
        s.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        with torch.cuda.graph(g, stream=s):
            work()
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_refusals():
    say("refusals of the binding")
    x, g = torch.zeros((4, 64), dtype=BF, device=DEV), torch.ones(64, device=DEV)
    bad = [
        lambda: ng.ngram_add_norm(x.cpu(), g, EPS),
        lambda: ng.ngram_add_norm(x.half(), g, EPS),
        lambda: ng.ngram_add_norm(x[:, ::2], g, EPS),
        lambda: ng.ngram_add_norm(x.view(-1), g, EPS),
        lambda: ng.ngram_add_norm(x, g[:32], EPS),
        lambda: ng.ngram_add_norm(x, g, -1.0),
        lambda: ng.ngram_add_norm(x, g, EPS, quantise=False),
        lambda: ng.ngram_add_norm(x[:, :12].contiguous(), g, EPS),
        lambda: ng.ngram_add_norm(x, g, EPS, residual=x[:2].contiguous()),
        lambda: ng.ngram_add_norm(x, g, EPS, q_out=ng.Fp8.empty(4, 128)),
        lambda: ng.ngram_add_norm_grad(x, x, torch.ones(3, device=DEV), g),
        lambda: ng.ngram_add_norm_grad(x, x, torch.ones(4, device=DEV), g, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
        lambda: ng.ngram_quant_fp8(x, rows=False),
        lambda: ng.ngram_quant_fp8(x, q=ng.Fp8.empty(64, 4)),
        lambda: ng.ngram_quant_fp8(x, q=ng.Fp8.empty(4, 64), qt=ng.Fp8.empty(64, 4, block_rows=128)),
        lambda: ng.Fp8.empty(4, 64, block_rows=2),
        lambda: ng.Fp8(torch.empty(4, 64, dtype=torch.uint8, device=DEV), torch.empty(4, 4, dtype=torch.uint8, device=DEV), 4, 64),
    ]
    for f in bad:
        with pytest.raises(ng.NgramError):
            f()
