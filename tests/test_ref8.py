"""The plain forms of tests/ref8.py against independent sources: torch's E4M3
casts, differences of the forward, torch's AdamW, published splitmix64
outputs; and the rounding rules' properties.  No GPU."""
import json
import os

import numpy as np
import pytest

from tests import ref8

torch = pytest.importorskip("torch")


def test_decode_and_encode_equal_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = ref8.decode(codes)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(size=20000) * 10.0 ** rng.uniform(-4, 2, 20000), want[np.isfinite(want)],
                        (want[1:126] + want[:125]) / 2])
    x = x[np.abs(x) <= 448].astype(np.float32)
    assert np.array_equal(ref8.encode(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_exponent_is_the_smallest():
    a = np.float32([448.0, 448.0001, 449, 896, 224, 224.00002, 1e-30, 3e38, 1.75, 1.7500001]).astype(np.float64)
    e = ref8.exponent(a)
    assert np.all(a <= 448 * 2.0 ** e) and np.all(a > 448 * 2.0 ** (e - 1))
    assert ref8.exponent(np.zeros(1))[0] == 0 and ref8.exponent(np.float64([1e-44]))[0] == -126


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(2)
    n, d, eps, t = 3, 24, 1e-5, 1e-6
    s, gamma = rng.normal(size=(n, d)), rng.normal(size=d)
    dy, dsum = rng.normal(size=(n, d)), rng.normal(size=(n, d))

    def loss(s, gamma):
        r = 1 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
        return float((s * r * gamma * dy).sum() + (s * dsum).sum())

    r = 1 / np.sqrt((s * s).mean(axis=1) + eps)
    dx, dgamma, _, _ = ref8.add_norm_grad(dy, s, r, gamma, dsum)
    for i in range(n):
        for j in range(d):
            e = np.zeros((n, d))
            e[i, j] = t
            assert abs((loss(s + e, gamma) - loss(s - e, gamma)) / (2 * t) - dx[i, j]) < 1e-6
    for j in range(d):
        e = np.zeros(d)
        e[j] = t
        assert abs((loss(s, gamma + e) - loss(s, gamma - e)) / (2 * t) - dgamma[j]) < 1e-6


def test_adamw_equals_torch():
    rng = np.random.default_rng(3)
    h = {"lr": 1e-2, "beta1": 0.8, "beta2": 0.95, "eps": 1e-6, "weight_decay": 0.1}
    p = rng.normal(size=50)
    q = torch.nn.Parameter(torch.from_numpy(p.copy()))
    opt = torch.optim.AdamW([q], lr=h["lr"], betas=(h["beta1"], h["beta2"]), eps=h["eps"], weight_decay=h["weight_decay"])
    m, v = np.zeros(50), np.zeros(50)
    for step in range(1, 8):
        g = rng.normal(size=50)
        q.grad = torch.from_numpy(g.copy())
        opt.step()
        p, m, v = ref8.adamw(p, g, m, v, h, step)
        assert np.allclose(p, q.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_splitmix64_equals_published_outputs():
    golden = json.load(open(os.path.join(os.path.dirname(__file__), "golden", "splitmix64_vectors.json")))
    gamma = int(golden["gamma"], 16)
    for seed, want in ((0, [int(x, 16) for x in golden["state0_first3"]]), (golden["rosetta_seed"], golden["rosetta_first5"])):
        states = np.array([(seed + i * gamma) & ref8.MASK for i in range(len(want))], dtype=np.uint64)
        assert [int(x) for x in ref8.splitmix64(states)] == want


@pytest.mark.parametrize("positive", [False, True])
def test_random_rounding_is_unbiased_and_bounded(positive):
    rng = np.random.default_rng(4)
    x = np.abs(rng.normal(size=(1, 128))) * 10.0 ** rng.uniform(-3, 0, (1, 128))
    x[0, 0] = 448.0
    trials = np.concatenate([ref8.pack_state(x, rng.integers(0, 1 << 20, x.shape), positive)[2] for _ in range(4000)])
    step = ref8.step_at(x[0])
    assert np.all(np.abs(trials - x) < step)
    # a mean of 4000 draws of variance <= step^2 / 4 (and a bias below 2^-20 step), six standard deviations
    free = x[0] > 2.0 ** -9 if positive else np.ones(128, bool)
    assert np.all(np.abs(trials.mean(axis=0) - x[0])[free] <= (6 * 0.5 / np.sqrt(4000) + 2.0 ** -20) * step[free])
    if positive:
        assert np.all(trials > 0)
