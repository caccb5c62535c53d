"""The gradient's buffer of a distillation may be the logits' own or share no byte with them: workgroups read
a row's logits more than once, while others write theirs."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402

EINVAL = -1
A = 0x100000            # a fake, aligned device address (never dereferenced)


def args(dtype, n, V, ld):
    return ctypes.byref(ng._DistillArgs(A, 4 * A, 5 * A, None, n, V, ld, 5, dtype, dtype, 1.0))


def message(dtype, n, V, ld, dz, dld):
    """Of a call whose workspace is missing, which is looked at last."""
    rc = ng.lib().ngram_distill(args(dtype, n, V, ld), 6 * A, None, None, 1.0, dz, dld, None, 0, None)
    assert rc == EINVAL
    return ng.lib().ngram_last_error().decode()


# (rows, tokens, distance of logits' rows, elements from the logits to the gradient, distance of its rows)
SHARED = [(4, 100, 100, 1, 100), (4, 100, 100, -1, 100), (4, 100, 100, 100, 100), (4, 100, 100, 399, 100), (4, 100, 100, -399, 100),
          (4, 100, 200, 50, 200), (4, 100, 200, 99, 200), (4, 100, 200, 101, 200), (4, 100, 250, 151, 250), (4, 100, 250, -151, 250),
          (4, 100, 200, 100, 250), (4, 100, 200, 100, 100), (1, 100, 100, 8, 100), (1, 100, 1000, 99, 1000), (3, 1, 2, 2, 2),
          (1 << 30, 1 << 30, 1 << 50, 8, 1 << 50)]
APART = [(4, 100, 100, 0, 100), (4, 100, 100, 400, 100), (4, 100, 100, -400, 100), (4, 100, 200, 100, 200), (4, 100, 250, 150, 250),
         (4, 100, 250, 100, 250), (4, 100, 250, -100, 250), (4, 100, 250, 350, 250), (4, 100, 200, 700, 300), (1, 100, 1000, 100, 1000),
         (4, 100, 200, -400, 100), (3, 1, 2, 1, 2)]


@pytest.mark.parametrize("dtype", [0, 1])
def test_partial_overlap_is_refused(dtype):
    size = 4 if dtype == 0 else 2
    for n, V, ld, at, dld in SHARED:
        assert "overlap" in message(dtype, n, V, ld, A + at * size, dld), (n, V, ld, at, dld)
        rc = ng.lib().ngram_distill_grad(args(dtype, n, V, ld), 6 * A, None, 1.0, A + at * size, dld, None)
        assert rc == EINVAL and "overlap" in ng.lib().ngram_last_error().decode()
    for n, V, ld, at, dld in APART:
        assert "workspace" in message(dtype, n, V, ld, A + at * size, dld), (n, V, ld, at, dld)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V", [(5, 1003), (3, 70001), (130, 70001)])
def test_interleaved_rows(n, V, dtype):
    """Rows of logits and gradient in turn in one buffer share no byte."""
    print(f"[case] distill interleaved {n} x {V} {dtype}", flush=True)
    g = torch.Generator(device="cuda:0").manual_seed(V)
    both = torch.randn((n, 2, V), generator=g, device="cuda:0").to(dtype)
    z = both[:, 0].clone()
    t, ids = torch.randn((n, 7), generator=g, device="cuda:0"), torch.randint(0, V, (n, 7), generator=g, device="cuda:0", dtype=torch.int32)
    lse = torch.logsumexp(t, dim=1) + 0.3
    want = ng.ngram_distill(z, t, ids, 1.0, lse, grad=True, keep_stats=True)
    got = ng.ngram_distill(both[:, 0], t, ids, 1.0, lse, dlogits_out=both[:, 1], keep_stats=True)
    assert torch.equal(got.loss, want.loss) and torch.equal(both[:, 1], want.dlogits) and torch.equal(both[:, 0], z)
    ng.ngram_distill_grad(both[:, 0], t, ids, got.stats, 1.0, lse, dlogits_out=both[:, 1])
    assert torch.equal(both[:, 1], ng.ngram_distill_grad(z, t, ids, got.stats, 1.0, lse)) and torch.equal(both[:, 0], z)
