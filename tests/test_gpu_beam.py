"""ngram_beam_step and ngram_beam_reorder on the GPU.

Tokens, parents, histories and marks equal the float64 search's: the seeds'
candidates lie further apart than fp32 sums of exp can move them (checked),
or tie exactly, which goes to the lowest place.  A score is off by the relative
error of its row's sum (ref_vocab.sum_error) and its own rounding."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref_vocab as ref  # noqa: E402
from tests.ref_vocab import U  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32, dev  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu


def inputs(rng, batch, beams, V, dtype):
    rows = batch * beams
    x = (rng.normal(size=(rows, V)) * 2).astype(np.float32)
    if dtype == BF:
        x = ref.bf16(x)
    return dict(logits=x, scores=(-12 * rng.random(rows)).astype(np.float32), tokens=rng.integers(0, V, rows).astype(np.int32),
                history=rng.integers(0, V, (rows, 2)).astype(np.int32), finished=rng.random(rows) < 0.15)


def on_gpu(a, dtype):
    return dict(logits=dev(a["logits"], dtype), scores=dev(a["scores"]), tokens=dev(a["tokens"]), history=dev(a["history"]),
                finished=dev(a["finished"]))


def check(a, out, beams, end, least_gap=True):
    want = ref.beam_step(a["logits"], a["scores"], beams, a["tokens"], a["history"], a["finished"], end)
    with np.errstate(all="ignore"):
        err = np.nan_to_num(ref.sum_error(a["logits"], 1.0), nan=0.0).max()
    if least_gap:
        assert want["gap"] > 2 * err + 1e-12, "the seed's candidates lie too close"
    for k in ("tokens", "parents", "history", "finished"):
        got = getattr(out, k)
        assert np.array_equal(got.cpu().numpy(), want[k]), k
    got, s = out.scores.double().cpu().numpy(), want["scores"]
    live = np.isfinite(s)
    assert np.array_equal(np.isfinite(got), live) and np.all(np.isneginf(got[~live]))
    assert np.all(np.abs(got[live] - s[live]) <= err + 2 * U * np.abs(s[live]) + err * 0.01)
    return want


SHAPES = [(1, 1, 1), (1, 1, 1000), (1, 2, 1), (3, 4, 3), (2, 5, 2), (2, 4, 50257), (1, 4, 151936), (5, 3, 4099), (1, 32, 700), (40, 8, 1003),
          (3, 32, 8193), (2, 7, 20001), (300, 4, 513), (1, 32, 151936), (1, 17, 70001)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,beams,V", SHAPES)
def test_step(batch, beams, V, dtype):
    say(f"beam step {batch} x {beams} x {V} {dtype}")
    a = inputs(np.random.default_rng(batch + 10 * beams + V), batch, beams, V, dtype)
    end = min(2, V - 1)
    g = on_gpu(a, dtype)
    out = ng.ngram_beam_step(g["logits"], g["scores"], beams, g["tokens"], g["history"], g["finished"], end)
    check(a, out, beams, end)


def test_ties_go_to_the_lowest_place():
    """Few distinct logits, equal rows with equal scores, -0 beside 0, and everything equal."""
    say("beam ties")
    rng = np.random.default_rng(5)
    for batch, beams, V, values in ((3, 4, 5000, 3), (2, 8, 9001, 2), (1, 32, 777, 1), (2, 16, 40000, 2)):
        row = rng.integers(0, values, (batch, 1, V)).astype(np.float32) * 0.5
        a = inputs(rng, batch, beams, V, F32)
        a["logits"] = np.broadcast_to(row, (batch, beams, V)).reshape(-1, V).copy()
        zero = a["logits"] == 0
        a["logits"][zero & (rng.random(zero.shape) < 0.5)] = -0.0
        a["scores"] = np.repeat(np.float32(-1.5), batch * beams)
        a["finished"][:] = False
        for dtype in (F32, BF):
            g = on_gpu(a, dtype)
            out = ng.ngram_beam_step(g["logits"], g["scores"], beams, g["tokens"], g["history"], end_token=7)
            check(a, out, beams, 7, least_gap=False)


@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("beams", [1, 5, 32])
def test_sorted_logits(beams, order):
    """Rising logits pass the threshold at every vector."""
    say(f"beam sorted {order} {beams}")
    rng = np.random.default_rng(6)
    V = 30000
    a = inputs(rng, 2, beams, V, F32)
    x = np.linspace(-8, 8, V, dtype=np.float32)
    a["logits"] = np.stack([(x if order == "rising" else x[::-1]) + np.float32(0.37) * np.float32(r) for r in range(2 * beams)])
    a["finished"][:] = False
    # equal up to a shift, so equal distributions: the scores alone order the beams' candidates
    g = on_gpu(a, F32)
    out = ng.ngram_beam_step(g["logits"], g["scores"], beams, g["tokens"], g["history"], g["finished"], 3)
    want = ref.beam_step(a["logits"], a["scores"], beams, a["tokens"], a["history"], a["finished"], 3)
    err = ref.sum_error(a["logits"], 1.0).max()
    got = out.scores.double().cpu().numpy()
    assert np.all(np.abs(got - want["scores"]) <= 1.01 * err + 2 * U * np.abs(want["scores"]))
    if want["gap"] > 2 * err:
        assert np.array_equal(out.tokens.cpu().numpy(), want["tokens"])


def test_masks_and_dead_beams():
    say("beam masks")
    rng = np.random.default_rng(8)
    batch, beams, V = 6, 4, 3001
    for dtype in (F32, BF):
        a = inputs(rng, batch, beams, V, dtype)
        x, lowest = a["logits"], np.float32(torch.finfo(dtype).min)
        a["finished"][:] = False
        a["scores"][1:4] = -np.inf                      # a search that starts
        x[4:8] = -np.inf                                # a sequence without candidates
        x[8, 5], x[9, 7], x[10] = np.nan, np.inf, -np.inf
        x[12:16, 3:] = -np.inf                          # three tokens left
        x[16:20] = lowest                               # masked by the type's lowest value: a uniform row
        x[20, 10:], x[21, 10:] = lowest, -np.inf
        a["scores"][20], a["scores"][22] = np.nan, np.inf
        a["finished"][13], a["finished"][18] = True, True
        a["scores"][22] = -np.inf
        a["finished"][22] = True                        # a finished beam that is dead
        g = on_gpu(a, dtype)
        out = ng.ngram_beam_step(g["logits"], g["scores"], beams, g["tokens"], g["history"], g["finished"], 2)
        check(a, out, beams, 2, least_gap=False)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_and_unaligned_rows(dtype):
    say(f"beam strides {dtype}")
    rng = np.random.default_rng(9)
    batch, beams, V = 2, 3, 4001
    a = inputs(rng, batch, beams, V, dtype)
    plain = None
    for pad, skip in ((0, 0), (1, 1), (7, 3), (64, 5)):
        wide = torch.full((batch * beams, V + pad + skip), 50.0, dtype=dtype, device=DEV)
        wide[:, skip:skip + V] = dev(a["logits"], dtype)
        g = on_gpu(a, dtype)
        out = ng.ngram_beam_step(wide[:, skip:skip + V], g["scores"], beams, g["tokens"], g["history"], g["finished"], 2)
        check(a, out, beams, 2)
        plain = plain or out
        assert torch.equal(out.tokens, plain.tokens)


def test_in_place_and_optional_outputs():
    say("beam in place")
    a = inputs(np.random.default_rng(10), 4, 4, 2000, F32)
    g = on_gpu(a, F32)
    ws = ng.beam_step_workspace(4, 4, 2000)
    want = ng.ngram_beam_step(g["logits"], g["scores"], 4, g["tokens"], g["history"], g["finished"], 2)
    out = ng.BeamOut(g["scores"], g["tokens"], torch.empty(16, dtype=torch.int32, device=DEV), g["history"], g["finished"])
    ng.ngram_beam_step(g["logits"], g["scores"], 4, g["tokens"], g["history"], g["finished"], 2, out=out, workspace=ws)
    for x, y in zip(want, out):
        assert torch.equal(x, y)
    g = on_gpu(a, F32)
    few = ng.ngram_beam_step(g["logits"], g["scores"], 4, out=ng.BeamOut(torch.empty(16, device=DEV), None, out.parents, None, None))
    assert few.tokens is None and torch.all(few.scores[1:4] <= few.scores[:3])
    none = ng.ngram_beam_step(torch.empty(0, 50, device=DEV), torch.empty(0, device=DEV), 4)
    assert none.scores.shape == (0,) and none.finished is None


def test_step_in_a_graph_and_on_two_streams():
    """Replays with other inputs in the same buffers, eager work between them, and two graphs that share one workspace on one stream."""
    say("beam graph")
    batch, beams, V = 3, 4, 6001
    sets = [inputs(np.random.default_rng(20 + i), batch, beams, V, BF) for i in range(3)]
    g = on_gpu(sets[0], BF)
    ws = ng.beam_step_workspace(batch, beams, V, BF)
    step = lambda: ng.ngram_beam_step(g["logits"], g["scores"], beams, g["tokens"], g["history"], g["finished"], 2, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        step()
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = step()
            graphs.append((graph, out))
    torch.cuda.synchronize()
    for a in sets + sets[:1]:
        for k, v in on_gpu(a, BF).items():
            g[k].copy_(v)
        eager = step()
        for graph, out in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, out in graphs:
            for x, y in zip(eager, out):
                assert torch.equal(x, y)
    other = ng.ngram_beam_step(g["logits"], g["scores"], beams, g["tokens"], g["history"], g["finished"], 2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(eager, other):
        assert torch.equal(x, y)


# ---------------------------------------------------------------------------------------------------------------

def moved(t, parents, beams):
    p = parents.cpu().numpy().reshape(-1, beams)
    own = np.broadcast_to(np.arange(beams), p.shape)
    row = np.where((p < 0) | (p >= beams), own, p) + np.arange(p.shape[0])[:, None] * beams
    return t.cpu()[torch.from_numpy(row.reshape(-1))]


@pytest.mark.parametrize("batch,beams", [(1, 1), (1, 2), (3, 4), (2, 5), (7, 8), (2, 13), (1, 16), (3, 17), (2, 32)])
def test_reorder(batch, beams):
    say(f"reorder {batch} x {beams}")
    rng = np.random.default_rng(batch * 40 + beams)
    rows = batch * beams
    make = lambda *s, dtype=torch.uint8: torch.randint(0, 256, s, device=DEV).to(dtype)  # noqa: E731
    wide = make(rows, 40, 9, dtype=torch.int32)
    states = [make(rows, 1), make(rows, 3), make(rows, 16), make(rows, 4096), make(rows, 4100), make(rows, 16 * 300 + 8), make(rows, 2, dtype=torch.int32),
              make(rows, 11, 7, dtype=torch.float32), make(rows, 5000, dtype=torch.int64), make(rows, dtype=torch.int32), wide[:, :20], wide[:, 24:30],
              make(rows, 0), make(rows, 17)[:, 1:9]]
    parents = rng.integers(-1, beams + 1, rows).astype(np.int32)
    want = [moved(t, torch.from_numpy(parents), beams) for t in states]
    between = wide[:, 20:24].clone()
    ng.ngram_beam_reorder(ng.BeamStates(states), dev(parents), beams)
    for t, w in zip(states, want):
        assert torch.equal(t.cpu(), w), tuple(t.shape)
    assert torch.equal(wide[:, 20:24], between)


def test_reorder_many_states_and_nothing():
    say("reorder many")
    states = [torch.randint(0, 1000, (8, 5 + i), device=DEV) for i in range(150)]
    parents = torch.tensor([1, 0, 3, 3, 2, 2, 0, 1], dtype=torch.int32, device=DEV)
    want = [moved(t, parents, 4) for t in states]
    lists = ng.BeamStates(states)
    ng.ngram_beam_reorder(lists, parents, 4)
    assert all(torch.equal(t.cpu(), w) for t, w in zip(states, want))
    ng.ngram_beam_reorder(ng.BeamStates([]), parents, 4)
    ng.ngram_beam_reorder(ng.BeamStates([torch.empty(0, 5, device=DEV)]), parents[:0], 4)


def test_reorder_in_a_graph():
    say("reorder graph")
    t = torch.randint(0, 1000, (8, 5000), device=DEV)
    parents = torch.tensor([1, 0, 3, 3, 2, 2, 0, 1], dtype=torch.int32, device=DEV)
    states = ng.BeamStates([t])
    ng.ngram_beam_reorder(states, parents, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ng.ngram_beam_reorder(states, parents, 4)
    for seed in range(3):
        t.copy_(torch.randint(0, 1000, (8, 5000), device=DEV))
        parents.copy_(torch.randint(0, 4, (8,), device=DEV))
        want = moved(t, parents, 4)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(t.cpu(), want)
