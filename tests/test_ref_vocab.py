"""The float64 forms of tests/ref_vocab.py against torch in float64, differences and brute force."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import ref_vocab as ref  # noqa: E402


def test_bf16_rounding_is_torch_s():
    x = np.random.default_rng(0).normal(size=4096).astype(np.float32) * np.float32(10) ** np.arange(-20, 20).repeat(103)[:4096].astype(np.float32)
    assert np.array_equal(ref.bf16(x), torch.from_numpy(x).bfloat16().float().numpy())
    assert ref.half_step(np.array([1.0]), True)[0] == 2.0 ** -8 and ref.half_step(np.array([1.0]), False)[0] == 2.0 ** -24


def test_pack_and_values():
    rng = np.random.default_rng(1)
    q = rng.integers(0, 16, (3, 72)).astype(np.uint8)
    codes = ref.pack(q, 72)
    assert codes.shape == (3, 48) and np.array_equal(ref.unpack(codes, 72), q)
    s, z = rng.random((3, 4)), rng.integers(0, 16, (3, 4)).astype(np.uint8)
    v = ref.values4(codes, s, z, 72, 32)
    assert v[2, 71] == (int(q[2, 71]) - int(z[2, 2])) * s[2, 2] and v[0, 31] == (int(q[0, 31]) - int(z[0, 0])) * s[0, 0]


@pytest.mark.parametrize("asym", [True, False])
def test_quantised_values_are_near(asym):
    """Rounded scale and zero included, a value is off by at most a step (asymmetric: half for the zero, half its own; and
    what a bf16 scale takes off the ends: 15 steps of 2^-9)."""
    x = np.random.default_rng(2).normal(size=(5, 200)).astype(np.float32)
    for bf in (True, False):
        q, s, z = ref.quant4(x, 64, asym, bf)
        v = ref.values4(ref.pack(q, 200), s, z, 200, 64)
        step = s[:, np.arange(200) // 64].astype(np.float64)
        assert np.all(np.abs(v - x) <= step * (1.0 if asym else 0.5) * (1 + 15 * 2.0 ** -8))


@pytest.mark.parametrize("rest", [False, True])
def test_distill_gradient_by_autograd_and_differences(rest):
    rng = np.random.default_rng(3)
    n, V, k, T = 4, 23, 5, 1.7
    z, t = rng.normal(size=(n, V)) * 2, rng.normal(size=(n, k)) * 2
    ids = np.array([rng.permutation(V)[:k] for _ in range(n)])
    ids[1, 3:], ids[2, 4] = -1, ids[2, 0]
    lse = ref.log_sum(t / T) + 0.3 if rest else None
    w = np.array([1.0, 0.5, 2.0, 0.0])
    loss, stats, grad, _ = ref.distill(z, t, ids, T, lse, w, 0.7)
    zt = torch.from_numpy(z).requires_grad_()
    q = torch.log_softmax(zt / T, dim=1)
    total = 0
    for i in range(n):
        on = ids[i] >= 0
        tt = torch.from_numpy(t[i][on] / T)
        lp = tt - (lse[i] if rest else torch.logsumexp(tt, 0))
        p = lp.exp()
        one = (p * (lp - q[i, ids[i][on]])).sum()
        if rest:
            off = torch.ones(V, dtype=torch.bool)
            off[ids[i][on]] = False
            P = 1 - p.sum()
            one = one + P * (P.log() - torch.log(q[i][off].exp().sum()))
        assert abs(float(one.detach()) * T * T - loss[i]) < 1e-12
        total = total + one * T * T * w[i] * 0.7
    total.backward()
    assert np.allclose(zt.grad.numpy(), grad, rtol=0, atol=1e-12)
    for i, j in ((0, 3), (1, int(ids[1, 0])), (2, int(ids[2, 0]))):
        h = 1e-6
        up, down = z.copy(), z.copy()
        up[i, j] += h
        down[i, j] -= h
        d = sum(wi * 0.7 * (a - b) for wi, a, b in zip(w, ref.distill(up, t, ids, T, lse)[0], ref.distill(down, t, ids, T, lse)[0])) / (2 * h)
        assert abs(d - grad[i, j]) < 1e-7


def test_distill_edges():
    z = np.array([[0.0, 1.0, -np.inf, 2.0], [0.0, 0.0, 0.0, 0.0], [-np.inf] * 4, [0.0, 1.0, 2.0, 3.0]])
    t, ids = np.zeros((4, 2)), np.array([[2, 0], [-1, 9], [0, 1], [0, 3]])
    loss, _, grad, _ = ref.distill(z, t, ids, 1.0)
    assert loss[0] == np.inf and loss[1] == 0 and np.all(grad[1] == 0) and np.isnan(loss[2])
    # one listed token: its cross entropy
    one = ref.distill(z[3:], t[3:, :1], np.array([[3]]), 1.0)[0][0]
    assert abs(one - (np.log(np.exp(z[3]).sum()) - 3.0)) < 1e-14


def test_beam_step_is_an_exhaustive_search():
    """Three steps of a search that keeps everything are the sums over all sequences."""
    rng = np.random.default_rng(4)
    V, B = 3, 27
    table = rng.normal(size=(40, V))                         # logits by last token and step
    scores = np.full(B, -np.inf)
    scores[0] = 0.0
    paths = [[] for _ in range(B)]
    for step in range(3):
        logits = np.stack([table[step * 4 + (p[-1] if p else 3)] for p in paths])
        out = ref.beam_step(logits, scores, B)
        scores = out["scores"]
        paths = [paths[b] + [int(t)] if b >= 0 else [] for b, t in zip(out["parents"], out["tokens"])]
    want = {}
    for a in range(V):
        for b in range(V):
            for c in range(V):
                s, last = 0.0, 3
                for step, tok in enumerate((a, b, c)):
                    row = table[step * 4 + last]
                    s, last = s + row[tok] - np.log(np.exp(row).sum()), tok
                want[(a, b, c)] = s
    assert [tuple(p) for p in paths] == sorted(want, key=lambda k: -want[k])
    assert np.allclose(scores, sorted(want.values(), reverse=True))


def test_beam_step_edges():
    x = np.array([[0.0, 0.0, -np.inf], [np.nan, 0.0, 0.0], [5.0, 5.0, 5.0], [-np.inf] * 3])
    out = ref.beam_step(x, np.array([0.0, 0.0, -3.0, 0.0]), 4, tokens=[7, 8, 9, 6], history=[(1, 2), (3, 4), (5, 6), (0, 0)],
                        finished=[False, False, True, False], end=1)
    assert out["parents"].tolist() == [0, 0, 2, -1] and out["tokens"].tolist() == [0, 1, 1, -1]
    assert out["finished"].tolist() == [False, True, True, False] and out["history"].tolist() == [[2, 7], [2, 7], [6, 9], [-1, -1]]
    assert out["scores"][2] == -3.0 and out["scores"][3] == -np.inf
