"""AdamW where the second moment is below fp32's smallest normal number and eps
is smaller still: the update is m / sqrt(v), not m / eps.

Tolerances.  v' takes three roundings; below 2^-126 each is half of 2^-149 at
most, so sqrt(v') is off by at most 0.5 * 1.5 * 2^-149 / v' of itself (twice
that is allowed for the second order), beside the 12 u of an ordinary update."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref8  # noqa: E402
from tests.ref8 import U  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32, dev, host  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
H = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-30, "weight_decay": 0.0}
LEAST = 2.0 ** -142


def data(rng, rows, d):
    """Gradients and moments (m, root of v) with v' from 2^-142 to beyond 2^-126, in float32."""
    size = 10.0 ** rng.uniform(-21.3, -18.5, (rows, d))
    m, root = 0.3 * size * rng.normal(size=(rows, d)), np.maximum(size, 2.0 ** -70.9)
    return (size * rng.normal(size=(rows, d))).astype(np.float32), m.astype(np.float32), root.astype(np.float32)


def bound(want, m0, g, wv, step):
    parts = H["beta1"] * np.abs(m0) + (1 - H["beta1"]) * np.abs(g)
    update = H["lr"] / (1 - H["beta1"] ** step) * parts / (np.sqrt(wv / (1 - H["beta2"] ** step)) + H["eps"])
    return update * (12 * U + 1.5 * 2.0 ** -149 / wv) + 3 * U * np.abs(want)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("step", [1, 500])
def test_fp32_moments(whole, step):
    say(f"small second moments, fp32, whole={whole} step={step}")
    rng = np.random.default_rng(step)
    rows, d = 6, 520
    g, m, root = data(rng, rows, d)
    v = (root.astype(np.float64) ** 2).astype(np.float32)
    v.flat[7], g.flat[7] = 0.0, 0.0                     # an element without any gradient
    p, m_d, v_d = torch.zeros((rows, d), device=DEV), dev(m), dev(v)
    if whole:
        ng.ngram_adamw(ng.AdamWTensors([p], [dev(g)], [m_d], [v_d]), step=step, **H)
    else:
        ng.ngram_adamw_rows(p, m_d, v_d, torch.arange(rows, dtype=torch.int32, device=DEV), dev(g), step=step, **H)
    m0, v0, g0 = (x.astype(np.float64) for x in (m, v, g))
    want, wm, wv = ref8.adamw(np.zeros((rows, d)), g0, m0, v0, H, step)
    some = np.ones((rows, d), bool)
    some.flat[7] = False
    assert wv[some].min() >= LEAST and (wv < 2.0 ** -126).mean() > 0.5 and (wv > 2.0 ** -126).any()
    assert np.all(np.abs(host(v_d) - wv) <= 1.5 * 2.0 ** -149 + 5 * U * wv)
    near = bound(want[some], m0[some], g0[some], wv[some], step)
    assert np.all(np.abs(host(p)[some] - want[some]) <= near)


@pytest.mark.parametrize("whole", [True, False])
def test_8_bit_moments(whole):
    say(f"small second moments, 8 bits, whole={whole}")
    rng = np.random.default_rng(9)
    rows, d, step = 6, 640, 100
    g, m, root = data(rng, rows, d)
    (mc, ms), (vc, vs) = ref8.quant(m.astype(np.float64)), ref8.quant(root.astype(np.float64))
    vc = np.where(vc == 0, 1, vc).astype(np.uint8)
    nb = d // 128
    m0, r0 = ref8.values(mc, ms, d), ref8.values(vc, vs, d)
    p = torch.zeros((rows, d), device=DEV)
    state = [dev(x) for x in (mc, vc, ms[:, :nb], vs[:, :nb])]
    if whole:
        ng.ngram_adamw(ng.AdamWTensors([p], [dev(g)], [state[0]], [state[1]], [state[2]], [state[3]]), step=step, **H)
    else:
        ng.ngram_adamw_rows(p, state[0], state[1], torch.arange(rows, dtype=torch.int32, device=DEV), dev(g), m_scale=state[2],
                            v_scale=state[3], step=step, **H)
    g0 = g.astype(np.float64)
    want, _, wv = ref8.adamw(np.zeros((rows, d)), g0, m0, r0 ** 2, H, step)
    big = wv >= LEAST
    assert big.mean() > 0.9 and (wv[big] < 2.0 ** -126).mean() > 0.3
    assert np.all(np.abs(host(p)[big] - want[big]) <= bound(want[big], m0[big], g0[big], wv[big], step))
    codes, scales = state[1].cpu().numpy(), state[3].cpu().numpy()
    unit = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 128, axis=1)
    val, x = ref8.decode(codes) * unit, np.sqrt(wv)
    off = x * (8 * U + 1.5 * 2.0 ** -149 / wv)          # of the root, before it is rounded to one of its neighbours
    assert np.all(val > 0)
    assert np.all((np.abs(val - x) <= ref8.step_at((x + off) / unit) * unit * (1 + 2.0 ** -18) + off)[big])


@pytest.mark.parametrize("factor", [0.9, 1.1])
def test_eps_around_the_switch(factor):
    """From eps = 2^-39 / sqrt(1 - beta2^step) on the root of a v' below 2^-126 may be left out: one u of the update more."""
    say(f"eps beside small roots {factor}")
    rng = np.random.default_rng(3)
    rows, d = 6, 520
    g, _, _ = data(rng, rows, d)
    h = dict(H, eps=factor * 2.0 ** -39 / np.sqrt(1 - H["beta2"]))
    p, m, v = (torch.zeros((rows, d), device=DEV) for _ in range(3))
    ng.ngram_adamw(ng.AdamWTensors([p], [dev(g)], [m], [v]), step=1, **h)
    g0 = g.astype(np.float64)
    want, _, wv = ref8.adamw(np.zeros((rows, d)), g0, np.zeros((rows, d)), np.zeros((rows, d)), h, 1)
    update = h["lr"] * np.abs(g0) / (np.abs(g0) + h["eps"])
    assert np.all(np.abs(host(p) - want) <= 13 * U * update + 3 * U * np.abs(want) + 1e-44)


def test_bf16_parameters_and_gradients():
    """The update in a bf16 parameter: minus lr times the sign of the gradient at step 1, to within a bf16 step."""
    say("small second moments, bf16")
    g = torch.tensor([1e-20, -1e-20, 3e-19, -1e-18, 1e-10] * 30, device=DEV).to(BF)
    p = torch.zeros(150, dtype=BF, device=DEV)
    m, v = torch.zeros(150, dtype=F32, device=DEV), torch.zeros(150, dtype=F32, device=DEV)
    ng.ngram_adamw(ng.AdamWTensors([p], [g], [m], [v]), step=1, **H)
    assert torch.all((p.float() + 1e-3 * g.float().sign()).abs() <= 1e-3 * (2.0 ** -7 + 0.01))
