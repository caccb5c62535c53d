"""ngram_distill and ngram_distill_grad with the teacher's rest where listed and unlisted tokens are far
apart, against float64 in logarithms (Q itself may be no number there).

Tolerances.  S and S' are the relative errors of the sums of exp over all and over the unlisted tokens, each
relative to its own largest logit (ref_vocab.sum_error); log Q is formed in float64 from them.  loss / T^2:
S of log q and S + S' of log Q, times p and P (at most 1 together), and its rounding.  stats: log Q is off by S
+ S' and its rounding.  Gradient off the list, (Q - P) q': Q by S + S', its exponent (4 u |log Q|) and 8 u; q' by
S' and its exponent, 4 u (|x - m'| / T + |log sum'|), the logarithm (4 u of it) and 12 u of exp2, products
and the factor.  From given statistics the exponent is relative to the row's largest logit where log Q >= -64:
S, S', the roundings of log sum and log Q and of the exponent's parts, 8 u (|x - m| / T + |log sum| + |log Q|) in
all, and Q is off by S + S' + 2 u |log Q|; else it is as above.  On the list, q - p: as test_gpu_distill has it.  exp2
gives 0 below 2^-126, a bf16 exponent of up to 2^12 rounds by 2^-13 (test_gpu_distill_fills), and the result to its type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref_vocab as ref  # noqa: E402
from tests.ref_vocab import U  # noqa: E402
from tests.test_gpu_distill import gpu  # noqa: E402
from tests.test_gpu_distill_fills import SHAPES, rounded, rows_of, spread  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu

KINDS = [(s, T) for i, s in enumerate(SHAPES) for T in ((1.0, 2.0), (1.5, 4.0))[i % 2]]


def definition(a, scale):
    """loss, log Q, gradient, and the pieces that the bounds need, a row at a time."""
    z, T, n, V = np.asarray(a["z"], np.float64), a["T"], *a["z"].shape
    out = dict(loss=np.zeros(n), log_q=np.zeros(n), log_s=np.zeros(n), grad=np.zeros((n, V)), q=np.zeros((n, V)), own=np.zeros((n, V)),
               p=np.zeros((n, V)), off=np.ones((n, V), bool), F=np.zeros(n), P=np.zeros(n), m=np.zeros(n), m_off=np.full(n, -np.inf),
               l_off=np.zeros(n))
    for i in range(n):
        x, idx = z[i], a["ids"][i]
        idx_on = (idx >= 0) & (idx < V)
        off = out["off"][i]
        off[idx[idx_on]] = False
        m = x.max()
        log_s = np.log(np.exp((x - m) / T).sum())
        log_p = np.asarray(a["t"], np.float64)[i][idx_on] / T - float(a["lse"][i])
        p, w = np.exp(log_p), float(a["weight"][i]) * scale * T
        loss = (p * (log_p - ((x[idx[idx_on]] - m) / T - log_s))).sum()
        P, log_q, Q = max(0.0, 1.0 - p.sum()), -np.inf, 0.0
        if off.any() and x[off].max() > -np.inf:
            mo = x[off].max()
            e = np.where(off, np.exp((np.where(off, x, mo) - mo) / T), 0.0)
            log_q = (mo - m) / T + np.log(e.sum()) - log_s
            Q = np.exp(log_q)
            out["own"][i], out["m_off"][i], out["l_off"][i] = e / e.sum(), mo, np.log(e.sum())
            out["F"][i] = Q - P if P > 0 else Q
        if P > 0:
            loss += P * (np.log(P) - log_q)
        np.add.at(out["p"][i], idx[idx_on], p)
        out["q"][i] = np.exp((x - m) / T - log_s)
        out["grad"][i] = w * np.where(off, out["F"][i] * out["own"][i], out["q"][i] - out["p"][i])
        out["loss"][i], out["log_q"][i], out["log_s"][i], out["P"][i], out["m"][i] = loss * T * T, log_q, log_s, P, m
    return out


def check(a, dtype, loss, grad, stats, given, scale=0.5):
    d = definition(a, scale)
    z, T, w = np.asarray(a["z"], np.float64), a["T"], a["weight"][:, None] * scale * a["T"]
    S, S2 = ref.sum_error(z, 1 / T), ref.sum_error(np.where(d["off"], z, -np.inf), 1 / T)
    some = np.isfinite(d["log_q"])
    lq, ls = np.where(some, d["log_q"], 0.0), d["log_s"]
    got, inf = loss.double().cpu().numpy(), np.isposinf(d["loss"])
    assert np.array_equal(np.isposinf(got), inf) and np.isfinite(got[~inf]).all()
    err, lb = np.abs(got[~inf] - d["loss"][~inf]), T * T * (2 * S + S2)[~inf] * 1.01 + 2 * U * np.abs(d["loss"][~inf])
    assert np.all(err <= lb), (err / lb).max()
    st = stats.double().cpu().numpy()
    assert np.array_equal(st[:, 0], d["m"]) and np.all(np.abs(st[:, 1] - ls) <= S + U * np.abs(ls))
    assert np.array_equal(np.isneginf(st[:, 2]), ~some) and np.all(np.abs(st[some, 2] - lq[some]) <= (S + S2 + 2 * U * np.abs(lq))[some])
    with np.errstate(all="ignore"):
        gap = np.where(np.isneginf(z), 0.0, (d["m"][:, None] - z) / T)
        gap_off = np.where(d["off"] & ~np.isneginf(z), (np.where(some, d["m_off"], 0.0)[:, None] - z) / T, 0.0)
    Q = np.exp(lq) * some
    own_err = S2[:, None] + U * (4 * gap_off + 8 * np.abs(d["l_off"])[:, None] + 12)
    q_unc = Q * (S + S2 + U * (4 * np.abs(lq) + 8))
    if given:
        near = (lq >= -64.0 - 1e-3)[:, None]
        own_err = np.where(near, (S + S2)[:, None] + U * (8 * (gap + np.abs(ls)[:, None] + np.abs(lq)[:, None]) + 12), own_err)
    F = np.abs(d["F"])[:, None]
    off_b = w * d["own"] * (F * own_err + q_unc[:, None] + U * F)
    on_b = w * (d["q"] * (S[:, None] + U * (4 * gap + 8 * np.abs(ls)[:, None] + 12)) + 4 * U * d["p"])
    gb = np.where(d["off"], off_b, on_b) * 1.02 + 2.0 ** -126 * (1 + w * (1 + F))
    gb += (2.0 ** -13 * np.abs(d["grad"]) if dtype == BF else 0)
    gb += ref.half_step(np.abs(d["grad"]) + gb, dtype == BF)
    g = grad.double().cpu().numpy()
    err = np.abs(g - d["grad"])
    assert grad.dtype == dtype and np.all(err <= gb), (err / gb).max()
    # what the unlisted tokens share out is Q - P
    total, want = np.where(d["off"], g, 0.0).sum(axis=1), (w * np.where(some, d["F"], 0.0)[:, None])[:, 0]
    assert np.all(np.abs(total - want) <= np.where(d["off"], gb, 0.0).sum(axis=1) + 1e-12 * np.abs(want))


def every_way(a, dtype, n=0):
    at, wide = spread(a, n)
    have = a["z"].shape[0]
    g = gpu(wide, dtype, dtype)
    kw = dict(temperature=a["T"], teacher_lse=g["lse"])
    one = ng.ngram_distill(g["z"], g["t"], g["ids"], grad=True, weight=g["weight"], scale=0.5, keep_stats=True, **kw)
    fwd = ng.ngram_distill(g["z"], g["t"], g["ids"], keep_stats=True, **kw)
    dz = ng.ngram_distill_grad(g["z"], g["t"], g["ids"], fwd.stats, weight=g["weight"], scale=0.5, **kw)
    inplace = g["z"].clone()
    ng.ngram_distill_grad(inplace, g["t"], g["ids"], fwd.stats, weight=g["weight"], scale=0.5, dlogits_out=inplace, **kw)
    assert torch.equal(inplace, dz)
    inplace.copy_(g["z"])
    ng.ngram_distill(inplace, g["t"], g["ids"], weight=g["weight"], scale=0.5, dlogits_out=inplace, **kw)
    assert torch.equal(inplace, one.dlogits)
    for x in (one.loss, one.dlogits, one.stats, fwd.loss, fwd.stats, dz):
        assert torch.equal(x, x[:have][torch.from_numpy(at).to(DEV)])
    check(a, dtype, one.loss[:have], one.dlogits[:have], one.stats[:have], False)
    check(a, dtype, fwd.loss[:have], dz[:have], fwd.stats[:have], True)


GAPS = [0.0, 20.0, 60.0, 70.0, 80.0, 86.0, 90.0, 100.0, 300.0, 1000.0, 1e4, 1e6, 1e9, 1e20]


@pytest.mark.parametrize("shape,T", KINDS)
def test_unlisted_tokens_far_below(shape, T):
    """Unlisted logits below the listed ones by up to 1e20: the loss is finite and their gradient sums to Q - P."""
    dtype, V, n = shape
    say(f"distill rest {V} {dtype} T={T}")
    k = (9, 200)[V % 2]
    rng = np.random.default_rng(V + 5)
    a = rows_of(rng, rng.normal(size=(len(GAPS) + 3, V)) * 2, k, dtype, T, True)
    for i, gap in enumerate(GAPS):
        low = a["z"][i] - np.float32(gap)
        low[a["ids"][i]] = a["z"][i][a["ids"][i]]
        a["z"][i] = rounded(low, dtype)
    up = len(GAPS)
    for j, gap in enumerate((100.0, 1e4)):                          # the other way round
        a["z"][up + j][a["ids"][up + j]] -= np.float32(gap)
    a["ids"][up + 2] = a["ids"][up + 2][0]                          # one token in every place, far above
    a["t"][up + 2] -= np.float32(T * np.log(k))
    a["z"][up + 2] -= np.float32(500)
    a["z"][up + 2][a["ids"][up + 2]] = 3.0
    a["z"], a["t"] = rounded(a["z"], dtype), rounded(a["t"], dtype)
    every_way(a, dtype, n)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,k", [(300, 300), (1000, 999), (40, 30), (9, 9)])
def test_few_or_no_unlisted_tokens(V, k, dtype):
    say(f"distill rest {V} of which {k} listed {dtype}")
    rng = np.random.default_rng(V + k)
    a = rows_of(rng, rng.normal(size=(6, V)) * 2, k, dtype, 1.5, True)
    off = np.ones((6, V), bool)
    off[np.arange(6)[:, None], a["ids"]] = False
    for i, fill in ((1, -np.inf), (2, -1e9), (3, 50.0), (4, np.float32(torch.finfo(dtype).min))):
        a["z"][i][off[i]] = rounded(fill, dtype)
    every_way(a, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_list_with_its_tokens_twice(dtype):
    """Every listed token in two places: its chance counts once."""
    say(f"distill rest twice {dtype}")
    rng = np.random.default_rng(8)
    for V, k in ((4001, 10), (70001, 700), (40001, 130)):
        a = rows_of(rng, rng.normal(size=(3, V)) * 2, k, dtype, 1.0, True)
        half = k // 2
        a["ids"][:, half:2 * half] = a["ids"][:, :half]
        a["z"][1] -= 200
        a["z"][1][a["ids"][1]] += 200
        a["z"][2][a["ids"][2]] += 3
        a["z"] = rounded(a["z"], dtype)
        every_way(a, dtype)
