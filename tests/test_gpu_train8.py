"""The 8-bit operators together: the training example's layer, its gradients
against a float64 layer, and decoding."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("train_projected_fp8", os.path.join(ROOT, "examples", "train_projected_fp8.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_lowers_the_loss(ex):
    say("training")
    layer, losses = ex.train(steps=48, say=None)
    first, last = np.mean(losses[:8]), np.mean(losses[-8:])
    print(f"[loss] {first:.4f} -> {last:.4f}", flush=True)
    assert np.all(np.isfinite(losses)) and last < 0.6 * first
    for t in (layer.table, layer.e1):
        assert torch.isfinite(t.p.float()).all() and torch.any(t.v > 0)


def test_layer_gradients_against_float64(ex):
    """The layer's gradients against autograd of the same layer in float64.  Quantising to E4M3 rounds by at
    most 2^-4 of a value; over sums of independent roundings the gradients differ by about 2^-4 / sqrt(3) = 3.6% of
    their size for each quantised factor, two a product, and two products in a row: below 15%."""
    say("layer gradients")
    layer = ex.Layer(R=3000, V=300, d=136, d_out=264, seed=3)
    n = 512
    tokens, offsets = ex.batch(layer.V, n, 4, 5)
    stream = torch.randn((n, layer.d), device="cuda:0").to(torch.bfloat16)
    dout = (torch.randn((n, layer.d_out), device="cuda:0") * 1e-2).to(torch.bfloat16)
    before = stream.clone()
    out = layer.forward(tokens, offsets, stream)
    dstream = layer.backward(dout)
    ids = layer.kept[1].cpu().long()
    leaf = lambda t: t.detach().cpu().double().requires_grad_()  # noqa: E731
    T, e1, W, gamma, P, s0 = (leaf(t) for t in (layer.table.p, layer.e1.p, layer.W_g, layer.gamma, layer.P, before))
    s = s0 + e1[tokens.cpu().long()] + W * T[ids].sum(dim=1)
    y = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + ex.EPS) * gamma
    want = y @ P.t()
    want.backward(dout.cpu().double())

    def gap(got, ref):
        return float(torch.linalg.norm(got.cpu().double() - ref) / torch.linalg.norm(ref))

    def dense(grad, size):
        rows, g, count = grad
        k = int(count.item())
        full = torch.zeros(size, dtype=torch.float64)
        full[rows[:k].cpu().long()] = g[:k].cpu().double()
        return full

    pairs = [("out", out, want.detach()), ("stream", dstream, s0.grad), ("P", layer.grads["P"], P.grad), ("gamma", layer.grads["gamma"], gamma.grad),
             ("W_g", layer.grads["W_g"], W.grad), ("table", dense(layer.sparse[0], T.shape), T.grad), ("e1", dense(layer.sparse[1], e1.shape), e1.grad)]
    for name, a, b in pairs:
        print(f"[gap] {name} {gap(a, b):.3f}", flush=True)
        assert gap(a, b) < 0.15, name


def test_decode_equals_the_batch(ex):
    """Token by token with history, and as one batch: the same 8-bit inputs, so the results differ by the product's
    summation order alone (both take the exact instruction here, rounded to bf16)."""
    say("decode")
    layer = ex.Layer(seed=4)
    tokens, _ = ex.batch(layer.V, 16, 1, 7)
    stream = torch.zeros((16, layer.d), dtype=torch.bfloat16, device="cuda:0")
    whole = layer.forward(tokens, torch.tensor([0, 16], dtype=torch.int32, device="cuda:0"), stream, keep=False).float()
    one = ex.decode(layer, tokens).float()
    assert torch.all((one - whole).abs() <= 2.0 ** -7 * whole.abs() + 1e-5)
