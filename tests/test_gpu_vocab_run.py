"""The vocabulary's operators together, as the example uses them: a search whose
scores are the log probabilities of what it wrote, eager and in a graph, and a
distillation step's gradients."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref_vocab as ref  # noqa: E402
from tests.ref_vocab import U  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("distill_and_search", os.path.join(ROOT, "examples", "distill_and_search.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_example_runs(ex):
    say("distillation")
    layer, losses = ex.train(steps=6, n=512, V=520, say=None)
    assert np.all(np.isfinite(losses)) and all(torch.isfinite(g).all() for g in layer.grads.values())


@pytest.mark.parametrize("beams,batch,V", [(4, 3, 520), (1, 2, 264), (7, 5, 1000), (32, 1, 520)])
def test_scores_are_the_log_probabilities_of_what_was_written(ex, beams, batch, V):
    say(f"search {batch} x {beams} x {V}")
    layer = ex.Layer(R=3000, V=V, d=136, d_out=V, seed=beams)
    layer.P.mul_(2.5)                               # distributions with peaks
    layer.P[ex.END].mul_(0.0)                       # and an end that is not too likely to be met
    first = torch.arange(3, 3 + batch, dtype=torch.int32, device=DEV)
    steps = 6
    search = ex.Search(layer, first, beams=beams)
    written, scores = (t.clone() for t in search.run(steps))
    assert torch.all(written[:, 0] == first.repeat_interleave(beams)) and torch.all(torch.isfinite(scores))
    by_sequence = scores.view(batch, beams)
    assert torch.all(by_sequence[:, 1:] <= by_sequence[:, :-1])
    rows = {(r // beams, *w) for r, w in enumerate(written.tolist())}
    assert len(rows) == batch * beams               # no sequence is kept twice
    # fed again, token by token, with histories written out from the sequences: the same logits, bit for bit, whose
    # log softmax in float64 adds up to the score; a score's rounding comes once a step
    total, bound = np.zeros(batch * beams), np.zeros(batch * beams)
    ended = np.zeros(batch * beams, bool)
    w = written.cpu().numpy()
    for i in range(steps):
        before = np.full((batch * beams, 2), ng.PAD_ID, np.int32)
        for h in (1, 2):
            if i - h >= 0:
                before[:, 2 - h] = w[:, i - h]
        z = search.logits(written[:, i].contiguous(), torch.from_numpy(before).to(DEV)).cpu().numpy()
        p = ref.log_softmax(z)[np.arange(batch * beams), w[:, i + 1]]
        assert np.all(w[ended, i + 1] == ex.END)
        total += np.where(ended, 0.0, p)
        bound += np.where(ended, 0.0, ref.sum_error(z, 1.0)) + 2 * U * np.abs(total)
        ended |= w[:, i + 1] == ex.END
    assert np.all(np.abs(total - scores.double().cpu().numpy()) <= bound)
    assert np.array_equal(ended, search.finished.cpu().numpy())


def test_a_wide_search_finds_the_best_sequence(ex):
    """Two steps with as many beams as tokens see every sequence of two: the best one is there, first."""
    say("exhaustive search")
    V = 32
    layer = ex.Layer(R=500, V=V, d=64, d_out=V, seed=5)
    search = ex.Search(layer, torch.tensor([3], dtype=torch.int32, device=DEV), beams=V, end=-1)
    search.out = search.out._replace(finished=None)
    search.finished = None
    written, scores = search.run(2)
    pad = torch.full((V, 2), ng.PAD_ID, dtype=torch.int32, device=DEV)
    one = ref.log_softmax(search.logits(torch.full((V,), 3, dtype=torch.int32, device=DEV), pad).cpu().numpy())[0]
    after = pad.clone()
    after[:, 1] = 3
    two = ref.log_softmax(search.logits(torch.arange(V, dtype=torch.int32, device=DEV), after).cpu().numpy())
    best = np.sort((one[:, None] + two).reshape(-1))[::-1][:V]
    assert np.all(np.abs(scores.double().cpu().numpy() - best) <= 1e-4)
    a, b = np.unravel_index(np.argmax(one[:, None] + two), (V, V))
    assert written[0].tolist() == [3, a, b]


def test_captured_search_is_the_eager_one(ex):
    """Replays with eager work between them, and a second search on the same layer."""
    say("search in a graph")
    layer = ex.Layer(R=3000, V=520, d=136, d_out=520, seed=9)
    layer.P.mul_(2.5)
    first = torch.tensor([4, 8, 15], dtype=torch.int32, device=DEV)
    eager, captured, other = (ex.Search(layer, first, beams=5) for _ in range(3))
    captured.capture()
    other.capture()
    for _ in range(5):
        a, b = eager.run(1), captured.run(1)
        torch.cuda.synchronize()
        c = other.run(1)
        for x, y, z in zip(a, b, c):
            assert torch.equal(x, y) and torch.equal(x, z)
    for x, y in zip(eager.out, captured.out):
        assert torch.equal(x, y)


def test_distilled_layer_gradients_against_float64(ex):
    """The gradients of the projection and of the hidden state behind it from the loss's gradient.  E4M3 rounds by at most
    2^-4 of a value, over sums of independent roundings about 2^-4 / sqrt(3) = 3.6% of the result for each quantised
    factor: two for P, the gradient's and the input's, and as many for dy: below 10%.  The loss's gradient itself,
    in bf16, is compared within its own bounds elsewhere; here it comes from float64 on the layer's own logits."""
    say("distilled gradients")
    layer, teacher = ex.Layer(R=3000, V=264, d=136, d_out=264, seed=3), ex.Layer(R=3000, V=264, d=136, d_out=264, seed=4)
    n, T = 512, 2.0
    tokens, offsets = ex.batch(layer.V, n, 4, 5)
    values, ids, lse = ex.teacher_lists(teacher, tokens, offsets, k=16, temperature=T)
    stream = torch.zeros((n, layer.d), dtype=torch.bfloat16, device=DEV)
    logits = layer.forward(tokens, offsets, stream)
    z = logits.float().cpu().numpy()
    out = ng.ngram_distill(logits, values, ids, T, lse, scale=1.0 / n, dlogits_out=logits)
    layer.backward(out.dlogits)
    loss, _, grad, _ = ref.distill(z, values.cpu().numpy(), ids.cpu().numpy(), T, lse.cpu().numpy(), None, 1.0 / n)
    # fp32 sums of some 264 terms, and a softmax at T
    assert np.allclose(out.loss.cpu().numpy(), loss, rtol=2.0 ** -18, atol=2.0 ** -18)
    y = layer.kept[3].y.double().cpu().numpy()
    dP = grad.T @ y
    got = layer.grads["P"].double().cpu().numpy()
    assert np.linalg.norm(got - dP) <= 0.1 * np.linalg.norm(dP)
    assert all(torch.isfinite(g).all() for g in layer.grads.values())
