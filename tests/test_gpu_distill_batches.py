"""Every element of the gradient of batches that fill the card, in float64 on the same device: rows in
registers in every size of them, vectors read again, and the calls apart.

Tolerances are test_gpu_distill's (gradient without the rest; with it the unlisted tokens' are those of
test_gpu_distill_rest, which for these rows, with Q of order one, are q (3 S + the exponents' u)), a row's S the largest
of them.  Zeros in the gradient's place would be off by 16 bounds and more nearly everywhere, which the test looks at."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.ref_vocab import U  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu


def expected(z, t, ids, lse, weight, scale, T):
    """(loss, gradient, its bound without the result's rounding), float64."""
    n, V = z.shape
    x = z.double()
    m = x.max(dim=1, keepdim=True).values
    d = (m - x) / T
    e = torch.exp(-d)
    log_s = e.sum(dim=1, keepdim=True).log()
    q = e / e.sum(dim=1, keepdim=True)
    # ref_vocab.sum_error, of all tokens and (with the rest) of the unlisted ones: their largest logit is at most m, their sum
    # at least (1 - listed mass) of it
    term = (q * (4 * d + 6)).sum(dim=1, keepdim=True)
    S = U * (term + 3 * V / 256 + 40)
    at = ids.long()
    log_p = t.double() / T - (lse.double()[:, None] if lse is not None else torch.logsumexp(t.double() / T, dim=1, keepdim=True))
    p = log_p.exp()
    P = torch.zeros_like(x).scatter_add_(1, at, p)
    log_q = -d.gather(1, at) - log_s
    loss = (p * (log_p - log_q)).sum(dim=1)
    a, F = p.sum(dim=1, keepdim=True), None
    if lse is not None:
        off = torch.ones_like(x, dtype=torch.bool).scatter_(1, at, False)
        rest, Q = 1 - p.sum(dim=1, keepdim=True), (q * off).sum(dim=1, keepdim=True)
        assert rest.min() > 0 and Q.min() > 0.1
        loss = loss + (rest * (rest.log() - Q.log()))[:, 0]
        a = torch.where(off, 1 - rest / Q, 1.0)
        S = S / Q
        F = off * (2 * S + U * (8 * Q.log().abs() + 12))
    w = weight.double()[:, None] * scale * T
    err = S + U * (8 * (d + log_s.abs()) + 12)
    bound = w * (q * (a.abs() * err + (F if F is not None else 0)) + 4 * U * P) * 1.02
    return loss * T * T, w * (a * q - P), bound, T * T * (3 * S[:, 0]) * 1.01 + 2 * U * (loss * T * T).abs()


def half_step(x, dtype):
    e = torch.frexp(x.abs())[1].clamp(min=-125)
    return torch.ldexp(torch.ones_like(x), e - (9 if dtype == BF else 25))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype,V", [(BF, 9001), (BF, 30001), (BF, 50257), (BF, 99999), (BF, 151936), (BF, 170001), (F32, 8192), (F32, 24577), (F32, 90002)])
def test_every_element(dtype, V, rest):
    say(f"distill batch {V} {dtype} rest={rest}")
    n, k, T, scale = 260, 70, 2.0, 0.5
    g = torch.Generator(device=DEV).manual_seed(V + rest)
    z = (torch.randn((n, V), generator=g, device=DEV) * 2).to(dtype)
    ids = torch.randint(0, V, (n, k), generator=g, device=DEV, dtype=torch.int32)
    t = torch.randn((n, k), generator=g, device=DEV)
    weight = torch.rand(n, generator=g, device=DEV) + 0.5
    lse = torch.logsumexp(t / T, dim=1) + 0.5 if rest else None
    kw = dict(temperature=T, teacher_lse=lse)
    one = ng.ngram_distill(z, t, ids, grad=True, weight=weight, scale=scale, **kw)
    fwd = ng.ngram_distill(z, t, ids, keep_stats=True, **kw)
    dz = ng.ngram_distill_grad(z, t, ids, fwd.stats, weight=weight, scale=scale, **kw)
    for at in range(0, n, 65):
        cut = slice(at, at + 65)
        loss, want, bound, lb = expected(z[cut], t[cut], ids[cut], lse[cut] if rest else None, weight[cut], scale, T)
        bound = bound + (2.0 ** -13 * want.abs() if dtype == BF else 0)
        bound = bound + half_step(want.abs() + bound, dtype)
        assert torch.all((want.abs() > 16 * bound).sum(dim=1) > V - 2 * k)      # zeros would not pass
        for got in (one, fwd):
            err = (got.loss[cut].double() - loss).abs()
            assert torch.all(err <= lb), (err / lb).max()
        for got in (one.dlogits, dz):
            err = (got[cut].double() - want).abs()
            assert torch.all(err <= bound), (err / bound).max()
