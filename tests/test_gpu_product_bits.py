"""What a result of ngram_project_fp8 keeps of small products beside large ones,
as include/ngram.h states it: a bf16 result of more than 32 rows takes the
products of eight consecutive columns as multiples of 2^(E - 13), cut towards
zero, E the largest sum of the two codes' exponents (a subnormal code's is
-6); everything else is exact to fp32.

Tolerances.  A group of eight is off by less than 8 * 2^(E - 13); fp32 sums
add 2 (K + 8) u of the sum of absolute terms, doubled for truncating adders;
a bf16 result half a step."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref8  # noqa: E402
from tests.ref8 import U  # noqa: E402
from tests.test_gpu_norm8 import BF, F32, dev  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu

# (m, n): 64 x 64, 128 x 128, 256 x 256 and 256 x 320 tiles over one block of 128 columns
TILES = [(100, 136), (1000, 1032), (2000, 4104), (4100, 4104)]


def code(x):
    return (ref8.code_of(np.abs(x)) | np.where(x < 0, 0x80, 0)).astype(np.uint8)


def matrix(codes, scales=None):
    rows, k = codes.shape
    if scales is None:
        scales = np.full((rows, ref8.scale_cols(k)), 127, dtype=np.uint8)
    return ng.Fp8(dev(codes), dev(scales), rows, k)


def exponents(codes):
    """The exponent fields of codes, -6 for subnormal codes."""
    return np.maximum((codes.astype(np.int64) >> 3) & 15, 1) - 7


@pytest.mark.parametrize("m,n", TILES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_products_from_a_unit_on_are_kept(m, n, sign):
    """+2^16 and -2^16 cancel in a group beside one product 2^e: 2^e >= 2^(16 - 13) is kept, a smaller one cut to zero."""
    say(f"kept and cut products {m} x {n} {sign}")
    a, b = np.zeros((m, 128)), np.zeros((n, 128))
    a[:, [40, 42]], b[:, [40, 42]] = [256.0, -256.0], 256.0
    x, y = np.arange(m) % 15 - 6, np.where(np.arange(n) % 2 == 0, 8, -6)
    a[:, 45], b[:, 45] = sign * 2.0 ** x, 2.0 ** y
    product = sign * 2.0 ** (x[:, None] + y[None, :])
    got = ng.ngram_project_fp8(matrix(code(a)), matrix(code(b)), dtype=BF).double().cpu().numpy()
    assert np.array_equal(got, np.where(np.abs(product) >= 2.0 ** 3, product, 0.0))
    exact = ng.ngram_project_fp8(matrix(code(a)), matrix(code(b)), dtype=F32).double().cpu().numpy()
    assert np.all(np.abs(exact - product) <= 2 * 136 * U * 2.0 ** 17)
    few = ng.ngram_project_fp8(matrix(code(a[:32])), matrix(code(b)), dtype=BF).double().cpu().numpy()
    assert np.all(np.abs(few - product[:32]) <= ref8.bf16_half_step(product[:32]) + 2 * 136 * U * 2.0 ** 17)


@pytest.mark.parametrize("m,n", TILES)
def test_other_groups_are_kept(m, n):
    """The same beside large products of another group of eight: nothing is cut down to 2^-8 of fp32's last place."""
    say(f"groups apart {m} x {n}")
    a, b = np.zeros((m, 128)), np.zeros((n, 128))
    a[:, [40, 42]], b[:, [40, 42]] = [256.0, -256.0], 256.0
    x = np.arange(m) % 12 - 3
    a[:, 48], b[:, 48] = 2.0 ** x, 1.0
    got = ng.ngram_project_fp8(matrix(code(a)), matrix(code(b)), dtype=BF).double().cpu().numpy()
    assert np.array_equal(got, np.repeat(2.0 ** x[:, None], n, axis=1))


@pytest.mark.parametrize("spread", [0.5, 2.0, 3.0])
@pytest.mark.parametrize("m,n,k", [(100, 136, 1032), (1000, 1032, 392), (2000, 4104, 128), (4100, 4104, 392)])
def test_bound(m, n, k, spread):
    """Random codes over many powers of two, subnormal ones among them, on a sample of the result."""
    say(f"bound {m} x {n} x {k} spread {spread}")
    rng = np.random.default_rng(m + k)
    draw = lambda r: ref8.quant(np.exp(spread * rng.normal(size=(r, k))) * rng.choice([-1, 1], (r, k)))  # noqa: E731
    a, b = draw(m), draw(n)
    got = ng.ngram_project_fp8(ng.Fp8(dev(a[0]), dev(a[1]), m, k), ng.Fp8(dev(b[0]), dev(b[1]), n, k), dtype=BF)
    rows, cols = np.sort(rng.permutation(m)[:64]), np.sort(rng.permutation(n)[:128])
    (ac, asc), (bc, bsc) = (a[0][rows], a[1][rows]), (b[0][cols], b[1][cols])
    av, bv = ref8.values(ac, asc, k), ref8.values(bc, bsc, k)
    want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
    cut = np.zeros_like(want)
    for at in range(0, ac.shape[1], 8):
        ea, eb = exponents(ac[:, at:at + 8]), exponents(bc[:, at:at + 8])
        top = (ea[:, None] + eb[None]).max(axis=2)
        scale = asc[:, at // 128].astype(int)[:, None] + bsc[:, at // 128].astype(int)[None] - 254
        cut += 2.0 ** (top + scale - 10)
    err = np.abs(got[dev(rows)][:, dev(cols)].double().cpu().numpy() - want)
    assert np.all(err <= ref8.bf16_half_step(want) * (1 + 2.0 ** -6) + cut + 2 * (k + 8) * U * size)


@pytest.mark.parametrize("outlier", [1, 30, 1000])
def test_the_norm_of_the_error_is_the_roundings(outlier):
    """With an outlier column too: the error's norm is at most 1% above that of rounding the exact result to bf16."""
    say(f"norm of the error, outlier {outlier}")
    rng = np.random.default_rng(outlier)
    m, n, k = 300, 264, 2560
    x = rng.normal(size=(m, k))
    x[:, 77] *= outlier
    a, b = ref8.quant(x), ref8.quant(rng.normal(size=(n, k)))
    want = ref8.values(*a, k) @ ref8.values(*b, k).T
    got = ng.ngram_project_fp8(ng.Fp8(dev(a[0]), dev(a[1]), m, k), ng.Fp8(dev(b[0]), dev(b[1]), n, k), dtype=BF).double().cpu().numpy()
    rounding = np.linalg.norm(ref8.bf16(want.astype(np.float32)) - want)
    assert np.linalg.norm(got - want) <= 1.01 * rounding
