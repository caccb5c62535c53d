"""ngram_distill and ngram_distill_grad where logits hold large finite numbers: mask fills over whole
runs of tokens and rows far from zero, through every kernel, against float64.

Tolerances are test_gpu_distill's, whose derivation does not use the logits' size: only differences to the
row's largest logit enter it, and a fill adds 0 to the sums on both sides.  A result below 2^-126 may be 0,
since exp2 gives no subnormal numbers: q is off by up to 2^-126 more, and the gradient by weight * scale * T * |a|
times that (or by 2^-126, where the factor is part of the exponent).  A bf16 gradient's exponent x c - K takes K =
m c + L below 2^12, rounded to fp32 once: half a step below 2^12 is 2^-13, and 2^(2^-13) - 1 is below 2^-13 (2^-13
ln 2 and a part in 10^4), so a q is off by 2^-13 of itself more."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref_vocab as ref  # noqa: E402
from tests.test_gpu_distill import bounds, check, gpu  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32, dev  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu

FILLS = [-1e4, -1e9, -1e10, -1e12, -1e20, -1e30]

# (type, tokens, rows): one launch with 4, 12 and 14 vectors a thread, rows in parts, one launch that reads the rest again
SHAPES = [(BF, 5003, 0), (BF, 30001, 0), (BF, 60001, 0), (BF, 70001, 0), (BF, 120001, 130),
          (F32, 5003, 0), (F32, 20001, 0), (F32, 30001, 0), (F32, 33001, 0), (F32, 60001, 130)]
KINDS = [(s, T, rest) for i, s in enumerate(SHAPES) for T in ((1.0, 1.5, 2.0, 4.0) if i % 5 in (0, 3) else ((1.0, 4.0), (2.0, 1.5))[i % 2])
         for rest in (False, True)]


def rounded(x, dtype):
    x = np.asarray(x, np.float32)
    return ref.bf16(x) if dtype == BF else x


def rows_of(rng, z, k, dtype, T, rest):
    """The teacher's side for logits z: k tokens a row, any of them."""
    n, V = z.shape
    ids = np.stack([rng.permutation(V)[:k] for _ in range(n)]).astype(np.int32)
    t = rounded(3 * rng.normal(size=(n, k)), dtype)
    lse = (ref.log_sum(np.asarray(t, np.float64) / T) + 0.02 + rng.random(n)).astype(np.float32) if rest else None
    return dict(z=rounded(z, dtype), t=t, ids=ids, lse=lse, weight=(rng.random(n) + 0.5).astype(np.float32), T=T)


def masked(rng, V, k, dtype, T, rest):
    """Every fill over the first tokens, a middle run, and all but the listed and a few others; and over none."""
    z = (rng.normal(size=(3 * len(FILLS) + 1, V)) * 2).astype(np.float32)
    a = rows_of(rng, z, k, dtype, T, rest)
    for i, fill in enumerate(FILLS):
        rows = 3 * i, 3 * i + 1, 3 * i + 2
        a["ids"][rows[0]] = V // 2 + rng.permutation(V // 2)[:k]
        a["ids"][rows[1]] = rng.permutation(V // 4)[:k]
        first, middle, most = a["z"][rows[0]], a["z"][rows[1]], a["z"][rows[2]]
        first[:V // 3] = rounded(fill, dtype)
        middle[V // 3:V // 3 + V // 2] = rounded(fill, dtype)
        keep = np.zeros(V, bool)
        keep[a["ids"][rows[2]]] = keep[rng.permutation(V)[:5]] = True
        keep[(a["ids"][rows[2], 0] + 1) % V] = True
        most[~keep] = rounded(fill, dtype)
    return a


def spread(a, n):
    """The rows over and over, to n of them."""
    have = a["z"].shape[0]
    at = np.arange(max(n, have)) % have
    return at, {k: (v[at] if isinstance(v, np.ndarray) else v) for k, v in a.items()}


def check_all(a, dtype, loss, grad, stats, scale=0.5):
    check(a, dtype, loss, None, stats, scale)
    if grad is not None:
        want = ref.distill(a["z"], a["t"], a["ids"], a["T"], a["lse"], a["weight"], scale)
        w = a["weight"][:, None] * scale * a["T"]
        gb = bounds(a, scale, dtype == BF, want)[1] + 2.0 ** -126 * np.maximum(1, w * np.abs(want[3]["a"]))
        gb = gb + (2.0 ** -13 * w * np.abs(want[3]["a"]) * want[3]["q"] if dtype == BF else 0)
        err = np.abs(grad.double().cpu().numpy() - want[2])
        assert grad.dtype == dtype and np.all(err <= gb), (err / gb).max()


def all_calls(a, dtype, n, see):
    """see(loss, gradient, statistics) of each way to the results for the distinct rows; the others repeat them."""
    have = a["z"].shape[0]
    at, wide = spread(a, n)
    g = gpu(wide, dtype, dtype)
    kw = dict(temperature=a["T"], teacher_lse=g["lse"])
    one = ng.ngram_distill(g["z"], g["t"], g["ids"], grad=True, weight=g["weight"], scale=0.5, keep_stats=True, **kw)
    fwd = ng.ngram_distill(g["z"], g["t"], g["ids"], keep_stats=True, **kw)
    dz = ng.ngram_distill_grad(g["z"], g["t"], g["ids"], fwd.stats, weight=g["weight"], scale=0.5, **kw)
    inplace = g["z"].clone()
    both = ng.ngram_distill(inplace, g["t"], g["ids"], weight=g["weight"], scale=0.5, dlogits_out=inplace, **kw)
    for x in (one.loss, one.dlogits, one.stats, fwd.loss, fwd.stats, dz):
        assert torch.equal(x, x[:have][torch.from_numpy(at).to(DEV)])
    assert torch.equal(both.loss, one.loss) and torch.equal(inplace, one.dlogits)
    see(one.loss[:have], one.dlogits[:have], one.stats[:have])
    see(fwd.loss[:have], dz[:have], fwd.stats[:have])


@pytest.mark.parametrize("shape,T,rest", KINDS)
def test_finite_fills(shape, T, rest):
    dtype, V, n = shape
    say(f"distill fills {V} {dtype} T={T} rest={rest}")
    a = masked(np.random.default_rng(V), V, 9, dtype, T, rest)
    all_calls(a, dtype, n, lambda loss, grad, stats: check_all(a, dtype, loss, grad, stats))


def shifted(rng, V, k, dtype, T, rest):
    """Rows far from zero: around 2^12, 2^19 and 2^20 of T / log2 e, both signs, and far beyond; one of equal fills."""
    unit = T * np.log(2)
    at = [s * x for x in (2 ** 12 * unit, 1e5, 2 ** 19 * 0.999 * unit, 2 ** 19 * 1.001 * unit, 2 ** 20 * unit, 1e6, 1e9, 1e10, 1e20, 1e30) for s in (1, -1)]
    z = np.stack([x + 10 * rng.normal(size=V) for x in at] + [np.full(V, -1e9)])
    return rows_of(rng, z, k, dtype, T, rest)


@pytest.mark.parametrize("shape,T,rest", KINDS)
def test_rows_far_from_zero(shape, T, rest):
    """Loss and statistics, and gradients of fp32."""
    dtype, V, n = shape
    say(f"distill far {V} {dtype} T={T} rest={rest}")
    a = shifted(np.random.default_rng(V + 1), V, 9, dtype, T, rest)
    all_calls(a, dtype, n, lambda loss, grad, stats: check_all(a, dtype, loss, grad if dtype == F32 else None, stats))


@pytest.mark.parametrize("shape,T,rest", [k for k in KINDS if k[0][0] == BF])
def test_bf16_gradients_far_from_zero(shape, T, rest):
    """Element by element: a gradient's exponent holds differences to the largest logit, whatever that is."""
    dtype, V, n = shape
    say(f"distill far gradient {V} {dtype} T={T} rest={rest}")
    a = shifted(np.random.default_rng(V + 2), V, 9, dtype, T, rest)
    # steps of bf16 at 2^12 T / log2 e are 16 and more; finer ones below
    for i, x in enumerate((1000, 2000, 2500, 2839, 2840, 3000, 5000, 20000)):
        a["z"][i] = rounded(x * T + 10 * np.random.default_rng(i).normal(size=V), dtype)
    all_calls(a, dtype, n, lambda loss, grad, stats: check_all(a, dtype, loss, grad, stats))


@pytest.mark.parametrize("dtype,V,n", [(BF, 5003, 0), (BF, 70001, 0), (F32, 5003, 0), (F32, 33001, 0), (F32, 60001, 130)])
@pytest.mark.parametrize("T", [2.0 ** -120, 1e-20, 1e-6, 1e-3, 1e3, 1e20, 1e37])
def test_extreme_temperatures(T, dtype, V, n):
    """log2 e / T over fp32's whole range: all of q on the largest logits, or none anywhere.  The loss carries T^2: above fp32's
    largest number (2^128 less half a step of 2^104) it rounds to infinity, and below 2^-126 its half step is 2^-150."""
    T = float(np.float32(T))
    say(f"distill T={T} {V} {dtype}")
    rng = np.random.default_rng(V + 3)
    a = rows_of(rng, rng.normal(size=(6, V)) * 2, 9, dtype, T, False)
    a["z"][1, :V // 3] = rounded(-1e10, dtype)
    a["z"][2] = rounded(1e10 + 1e9 * rng.normal(size=V), dtype)
    a["z"][3] = rounded(1e-3 * rng.normal(size=V), dtype)
    a["z"][4], a["t"][4] = 0.0, 0.0
    a["weight"][:] = np.float32(min(1.0, 1 / T))
    want = ref.distill(a["z"], a["t"], a["ids"], T, None, a["weight"], 0.5)
    lb = bounds(a, 0.5, dtype == BF, want)[0] + 2.0 ** -150

    def see(loss, grad, stats):
        got, most = loss.double().cpu().numpy(), 2.0 ** 128 - 2.0 ** 103
        sure = np.abs(want[0] - most) > lb
        assert np.array_equal(np.isposinf(got)[sure], want[0][sure] >= most)
        fine = np.isfinite(got)
        assert np.all(np.abs(got[fine] - want[0][fine]) <= lb[fine])
        check_all(a, dtype, None, grad, stats)
    all_calls(a, dtype, n, see)
