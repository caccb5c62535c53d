"""ngram_distill and ngram_distill_grad on the GPU against float64.

Tolerances.  S is the relative error of a row's sum of exp (ref_vocab.sum_error),
of the whole row and, with the teacher's rest, of the unlisted tokens.  The
teacher's side and the loss are float64, so loss / T^2 is off by S (times sum
p + rest, at most 1) from log q and by as much from log Q, and by its rounding to
fp32.  The gradient's q is off by S, by the fp32 log of the sum (its rounding,
and its product with log2 e, 2 u |log sum|), by the exponent (its difference,
product and sum: 4 u (|x - m| / T + |log sum|)) and by 4 u of exp2 and products;
the ratio P / Q by S twice, by log Q's rounding (u |log Q|) and 4 u; p by 2 u; then comes
the result's rounding."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref_vocab as ref  # noqa: E402
from tests.ref_vocab import U  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32, dev  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu


def inputs(rng, n, V, k, dtype, tdtype=None, rest=False, T=1.0):
    z = (rng.normal(size=(n, V)) * 2).astype(np.float32)
    ids = np.stack([rng.permutation(V)[:k] if k <= V else rng.integers(0, V, k) for _ in range(n)]).astype(np.int32)
    t = (3 * rng.normal(size=(n, k))).astype(np.float32)
    z[np.arange(n)[:, None], ids] += 2
    ids[rng.random((n, k)) < 0.1] = -1
    if n > 2:
        ids[n - 1] = V                              # nothing listed
        ids[n - 2, :] = ids[n - 2, 0]               # one token in every place
    z, t = (ref.bf16(v) if d == BF else v for v, d in ((z, dtype), (t, tdtype or dtype)))
    lse = (ref.log_sum(np.asarray(t, np.float64) / T) + 0.02 + rng.random(n)).astype(np.float32) if rest else None
    weight = (rng.random(n) + 0.5).astype(np.float32)
    weight[n // 2] = 0.0 if n > 1 else weight[0]
    return dict(z=z, t=t, ids=ids, lse=lse, weight=weight, T=T)


def bounds(a, scale, bf, want):
    """(of loss, of the gradient, of log Q)"""
    z, T = np.asarray(a["z"], np.float64), a["T"]
    loss, stats, grad, f = want
    S = ref.sum_error(z, 1 / T)
    if a["lse"] is not None:
        off = z.copy()
        for i, row in enumerate(a["ids"]):
            off[i, row[(row >= 0) & (row < z.shape[1])]] = -np.inf
        # relative to the row's maximum, not to the unlisted tokens' own
        S2 = S + ref.sum_error(off, 1 / T) + 4 * U * np.abs(z.max(axis=1) - np.maximum(off.max(axis=1), -1e30)) / T
    else:
        S2 = S
    lb = T * T * (S + S2) * 1.01 + 2 * U * np.abs(loss)
    m, ls = z.max(axis=1, keepdims=True), stats[:, 1:2]
    with np.errstate(all="ignore"):
        d = np.where(np.isneginf(z), 0, np.abs(z - m) / T)
    q_err = S[:, None] + U * (4 * (d + np.abs(ls)) + 4 * np.abs(ls) + 12)
    w = np.abs(a["weight"][:, None] * scale * T)
    ratio = (np.abs(f["ratio"]) * (2 * S2 + 2 * S + U * (np.abs(np.nan_to_num(stats[:, 2], neginf=0)) + 8)))[:, None]
    gb = w * (f["q"] * (np.abs(f["a"]) * q_err + ratio) + 4 * U * np.abs(f["p"])) * 1.02
    gb = gb + ref.half_step(np.abs(grad) + gb, bf)
    return lb, gb, S + S2 + 2 * U * np.abs(np.nan_to_num(stats[:, 2], neginf=0))


def gpu(a, dtype, tdtype):
    g = dict(z=dev(a["z"], dtype), t=dev(a["t"], tdtype), ids=dev(a["ids"]), weight=dev(a["weight"]))
    return g | {"lse": None if a["lse"] is None else dev(a["lse"])}


def check(a, dtype, got_loss, got_grad, got_stats=None, scale=1.0):
    want = ref.distill(a["z"], a["t"], a["ids"], a["T"], a["lse"], a["weight"], scale)
    lb, gb, qb = bounds(a, scale, dtype == BF, want)
    loss, stats, grad, _ = want
    if got_loss is not None:
        got, inf = got_loss.double().cpu().numpy(), np.isposinf(loss)       # a listed or an unlisted token without a chance
        assert np.array_equal(np.isposinf(got), inf)
        err = np.abs(got[~inf] - loss[~inf])
        assert np.all(err <= lb[~inf]), (err / lb[~inf]).max()
    if got_stats is not None:
        s = got_stats.double().cpu().numpy()
        assert np.array_equal(s[:, 0], np.asarray(a["z"], np.float64).max(axis=1))
        assert np.all(np.abs(s[:, 1] - stats[:, 1]) <= ref.sum_error(a["z"], 1 / a["T"]) + U * np.abs(stats[:, 1]))
        live = np.isfinite(stats[:, 2])
        assert np.all(np.abs(s[live, 2] - stats[live, 2]) <= qb[live])
    if got_grad is not None:
        assert got_grad.dtype == dtype
        err = np.abs(got_grad.double().cpu().numpy() - grad)
        assert np.all(err <= gb), (err / gb).max()


SHAPES = [(1, 1, 1), (1, 2, 2), (3, 7, 3), (5, 8, 1), (4, 1000, 10), (2, 151936, 64), (37, 5003, 33), (300, 257, 5), (9, 32003, 100), (3, 4099, 1024),
          (1100, 1001, 4), (6, 70000, 600), (2, 9, 300)]


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,V,k", SHAPES)
def test_loss_and_gradient(n, V, k, dtype, rest):
    """In one call, and apart; the gradient in a buffer of its own and in the logits' place."""
    say(f"distill {n} x {V}, {k} listed, {dtype} rest={rest}")
    T = [1.0, 2.0, 0.7, 4.0][(n + V + k) % 4]
    tdtype = F32 if (n + k) % 2 else dtype
    a = inputs(np.random.default_rng(n + V + k), n, V, k, dtype, tdtype, rest, T)
    g = gpu(a, dtype, tdtype)
    kw = dict(temperature=T, teacher_lse=g["lse"])
    scale = 0.25
    one = ng.ngram_distill(g["z"], g["t"], g["ids"], grad=True, weight=g["weight"], scale=scale, keep_stats=True, **kw)
    check(a, dtype, one.loss, one.dlogits, one.stats, scale)
    fwd = ng.ngram_distill(g["z"], g["t"], g["ids"], keep_stats=True, **kw)
    check(a, dtype, fwd.loss, None, fwd.stats)
    dz = ng.ngram_distill_grad(g["z"], g["t"], g["ids"], fwd.stats, weight=g["weight"], scale=scale, **kw)
    check(a, dtype, None, dz, None, scale)
    inplace = g["z"].clone()
    again = ng.ngram_distill_grad(inplace, g["t"], g["ids"], fwd.stats, weight=g["weight"], scale=scale, dlogits_out=inplace, **kw)
    assert again is inplace and torch.equal(inplace, dz)
    inplace = g["z"].clone()
    both = ng.ngram_distill(inplace, g["t"], g["ids"], weight=g["weight"], scale=scale, dlogits_out=inplace, **kw)
    assert torch.equal(both.loss, one.loss) and torch.equal(inplace, one.dlogits)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("n,V,k,dtype", [(2, 153897, 5, F32), (1, 153897, 200, F32), (1, 307793, 200, BF), (2, 307793, 5, BF)])
def test_long_rows_in_many_parts(n, V, k, dtype, rest):
    """Rows whose parts, rounded up to whole words of marks, are fewer than were asked for; the last vector is no whole one."""
    say(f"distill parts {n} x {V}, {k} listed, {dtype} rest={rest}")
    a = inputs(np.random.default_rng(n + V + k), n, V, k, dtype, None, rest, 1.5)
    g = gpu(a, dtype, dtype)
    kw = dict(temperature=1.5, teacher_lse=g["lse"])
    one = ng.ngram_distill(g["z"], g["t"], g["ids"], grad=True, weight=g["weight"], keep_stats=True, **kw)
    check(a, dtype, one.loss, one.dlogits, one.stats)
    inplace = g["z"].clone()
    both = ng.ngram_distill(inplace, g["t"], g["ids"], weight=g["weight"], dlogits_out=inplace, **kw)
    assert torch.equal(both.loss, one.loss) and torch.equal(inplace, one.dlogits)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_and_unaligned_rows(dtype):
    say(f"distill strides {dtype}")
    n, V, k = 5, 4001, 12
    a = inputs(np.random.default_rng(3), n, V, k, dtype, dtype, True, 1.5)
    g = gpu(a, dtype, dtype)
    for pad, skip, dpad, dskip in ((1, 1, 0, 0), (0, 0, 3, 2), (7, 3, 7, 3), (64, 5, 8, 1)):
        wide = torch.full((n, V + pad + skip), 90.0, dtype=dtype, device=DEV)
        wide[:, skip:skip + V] = g["z"]
        out = torch.full((n, V + dpad + dskip), 7.0, dtype=dtype, device=DEV)
        kw = dict(temperature=1.5, teacher_lse=g["lse"], weight=g["weight"])
        r = ng.ngram_distill(wide[:, skip:skip + V], g["t"], g["ids"], dlogits_out=out[:, dskip:dskip + V], keep_stats=True, **kw)
        check(a, dtype, r.loss, out[:, dskip:dskip + V].contiguous(), r.stats)
        assert torch.all(out[:, :dskip] == 7) and torch.all(out[:, dskip + V:] == 7) and torch.all(wide[:, :skip] == 90)
        out.fill_(7.0)
        ng.ngram_distill_grad(wide[:, skip:skip + V], g["t"], g["ids"], r.stats, dlogits_out=out[:, dskip:dskip + V], **kw)
        check(a, dtype, None, out[:, dskip:dskip + V].contiguous())
        assert torch.all(out[:, :dskip] == 7) and torch.all(out[:, dskip + V:] == 7)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_masks_and_strange_values(dtype, rest):
    say(f"distill masks {dtype} rest={rest}")
    n, V, k = 14, 3001, 6
    rng = np.random.default_rng(4)
    a = inputs(rng, n, V, k, dtype, dtype, rest, 1.0)
    a["weight"][:] = 1.0
    a["ids"] = np.stack([rng.permutation(V - 10)[:k] for _ in range(n)]).astype(np.int32)
    z, t, ids, lowest = a["z"], a["t"], a["ids"], np.float32(torch.finfo(dtype).min)
    free = np.ones((n, V), bool)
    free[np.arange(n)[:, None], ids] = False
    z[0][free[0]] = -np.inf                     # only listed tokens have a chance
    z[1, ids[1, 2]] = -np.inf                   # a listed token has none
    t[2, 1:] = -np.inf                          # one listed token counts
    t[3] = -np.inf                              # none counts
    z[4, 2000:] = -np.inf
    z[5] = lowest                               # uniform
    z[6, ::2] = lowest
    z[7], z[8, 9], z[9, 9] = -np.inf, np.nan, np.inf
    z[10, 5], a["weight"][10] = np.nan, 0.0     # weighs nothing
    t[11, 3] = np.nan
    z[12] += 60
    z[13, 7], ids[13] = 100.0, -1
    z, t = (ref.bf16(v) if dtype == BF else v for v in (z, t))
    a["z"], a["t"] = z, t
    ids[0][ids[0] >= 2000] %= 2000
    g = gpu(a, dtype, dtype)
    loss, stats, grad, f = ref.distill(z, t, ids, 1.0, a["lse"], a["weight"])
    r = ng.ngram_distill(g["z"], g["t"], g["ids"], teacher_lse=g["lse"], weight=g["weight"], grad=True, keep_stats=True)
    apart = ng.ngram_distill_grad(g["z"], g["t"], g["ids"], r.stats, teacher_lse=g["lse"], weight=g["weight"])
    got = r.loss.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(loss)) and np.array_equal(np.isposinf(got), np.isposinf(loss))
    assert np.isinf(loss[1]) and np.isnan(loss[[7, 8, 9, 10, 11]]).all() and (rest or loss[3] == got[3] == 0)
    keep = [i for i in range(n) if i not in (7, 8, 9, 10, 11)]
    cut = {k2: (v[keep] if isinstance(v, np.ndarray) else v) for k2, v in a.items()}
    fine = np.isfinite(loss[keep])
    small = {k2: (v[fine] if isinstance(v, np.ndarray) else v) for k2, v in cut.items()}
    check(small, dtype, r.loss[keep][torch.from_numpy(fine).to(DEV)], None)
    for dz in (r.dlogits, apart):
        check(cut, dtype, None, dz[keep])
        d = dz.float().cpu().numpy()
        assert np.all(d[10] == 0)
        for i in (7, 8, 9):
            assert np.isnan(d[i]).all()
        assert np.isnan(d[11]).any()


def test_cross_entropy_is_a_list_of_one():
    say("distill cross entropy")
    n, V = 50, 1003
    z = torch.randn(n, V, device=DEV)
    label = torch.randint(0, V, (n, 1), device=DEV, dtype=torch.int32)
    out = ng.ngram_distill(z, torch.zeros(n, 1, device=DEV), label, grad=True, scale=1 / n)
    ref_z = z.double().cpu().requires_grad_()
    want = torch.nn.functional.cross_entropy(ref_z, label[:, 0].long().cpu(), reduction="none")
    (want.sum() / n).backward()
    a = dict(z=z.cpu().numpy(), t=np.zeros((n, 1)), ids=label.cpu().numpy(), lse=None, weight=np.ones(n), T=1.0)
    lb, gb, _ = bounds(a, 1 / n, False, ref.distill(a["z"], a["t"], a["ids"], 1.0, None, a["weight"], 1 / n))
    assert np.all(np.abs(out.loss.double().cpu().numpy() - want.detach().numpy()) <= lb)
    assert np.all(np.abs(out.dlogits.double().cpu().numpy() - ref_z.grad.numpy()) <= gb)


def test_rows_do_not_depend_on_the_batch_s_other_rows_and_repeat():
    """The same call gives the same bits; a row among many gives what it gives among many others."""
    say("distill repeat")
    a = inputs(np.random.default_rng(6), 1200, 999, 8, BF, BF, True, 2.0)
    g = gpu(a, BF, BF)
    call = lambda s: ng.ngram_distill(g["z"][s], g["t"][s], g["ids"][s], 2.0, g["lse"][s], grad=True, weight=g["weight"][s], keep_stats=True)  # noqa: E731
    first, second, part = call(slice(0, 1200)), call(slice(0, 1200)), call(slice(64, 1200))
    for x, y, p in zip(first, second, part):
        assert torch.equal(x, y) and torch.equal(x[64:], p)


def test_nothing_to_do_and_guards():
    say("distill guards")
    empty = ng.ngram_distill(torch.empty(0, 50, device=DEV), torch.empty(0, 3, device=DEV), torch.empty(0, 3, dtype=torch.int32, device=DEV), grad=True)
    assert empty.loss.shape == (0,) and empty.dlogits.shape == (0, 50)
    for n, V in ((3, 1001), (2, 151936), (1100, 77)):
        for dtype in (BF, F32):
            z = torch.randn(n, V, device=DEV).to(dtype)
            t, ids = torch.randn(n, 4, device=DEV), torch.randint(0, V, (n, 4), device=DEV, dtype=torch.int32)
            flat = torch.full((n * V + 64,), 3.0, dtype=dtype, device=DEV)
            loss, stats = torch.full((n + 4,), 9.0, device=DEV), torch.full((3 * n + 4,), 9.0, device=DEV)
            ng.ngram_distill(z, t, ids, loss_out=loss, stats_out=stats, dlogits_out=flat[32:32 + n * V].view(n, V))
            assert torch.all(flat[:32] == 3) and torch.all(flat[32 + n * V:] == 3) and torch.all(loss[n:] == 9) and torch.all(stats[3 * n:] == 9)


def test_in_a_graph_and_on_another_stream():
    say("distill graph")
    n, V, k = 40, 5001, 9
    sets = [inputs(np.random.default_rng(30 + i), n, V, k, BF, BF, True, 1.0) for i in range(3)]
    g = gpu(sets[0], BF, BF)
    ws = ng.distill_workspace(n, V, k, BF)
    call = lambda **kw: ng.ngram_distill(g["z"], g["t"], g["ids"], 1.0, g["lse"], grad=True, weight=g["weight"], keep_stats=True, **kw)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        call(workspace=ws)
        for _ in range(2):                      # two graphs on one stream share a workspace
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = call(workspace=ws)
                dz = ng.ngram_distill_grad(g["z"], g["t"], g["ids"], out.stats, 1.0, g["lse"], weight=g["weight"])
            graphs.append((graph, out, dz))
    torch.cuda.synchronize()
    for a in sets + sets[:1]:
        for name, v in gpu(a, BF, BF).items():
            g[name].copy_(v)
        eager = call()
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        check(a, BF, eager.loss, eager.dlogits, eager.stats)
        for _, out, dz in graphs:
            for x, y in zip(eager, out):
                assert torch.equal(x, y)
            check(a, BF, None, dz)
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(eager, other):
        assert torch.equal(x, y)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype,V", [(BF, 30001), (BF, 50257), (BF, 99999), (BF, 151936), (BF, 170001), (F32, 8192), (F32, 24577), (F32, 90002)])
def test_batches_that_fill_the_card(dtype, V, rest):
    """Rows kept in registers, in every size of them and beyond; some rows against float64, all of them against the calls apart."""
    say(f"distill full batch {V} {dtype} rest={rest}")
    n, k = 260, 70
    some = [0, 1, 100, 130, 257, 258, 259]
    rng = np.random.default_rng(V)
    g = torch.Generator(device=DEV).manual_seed(V)
    z = (torch.randn((n, V), generator=g, device=DEV) * 2).to(dtype)
    a = inputs(rng, len(some), V, k, dtype, F32, rest, 2.0)
    z[some] = dev(a["z"], dtype)
    t, ids = torch.randn((n, k), generator=g, device=DEV), torch.randint(0, V, (n, k), generator=g, device=DEV, dtype=torch.int32)
    t[some], ids[some] = dev(a["t"]), dev(a["ids"])
    lse = torch.logsumexp(t / 2, dim=1) + 0.5 if rest else None
    weight = torch.rand(n, generator=g, device=DEV) + 0.5
    weight[some] = dev(a["weight"])
    if rest:
        lse[some] = dev(a["lse"])
    kw = dict(temperature=2.0, teacher_lse=lse)
    one = ng.ngram_distill(z, t, ids, grad=True, weight=weight, scale=0.5, keep_stats=True, **kw)
    check(a, dtype, one.loss[some], one.dlogits[some], one.stats[some], 0.5)
    fwd = ng.ngram_distill(z, t, ids, keep_stats=True, **kw)
    dz = ng.ngram_distill_grad(z, t, ids, fwd.stats, weight=weight, scale=0.5, **kw)
    # both within the bounds of one result, which for these rows are below 2^-14 (fp32 sums of some hundred terms a lane) and a bf16 step
    assert torch.allclose(one.loss, fwd.loss, rtol=0, atol=4 * 2 * 2.0 ** -14) and torch.allclose(one.stats, fwd.stats, rtol=2.0 ** -22, atol=2 * 2.0 ** -14)
    # listed tokens' q and p may cancel: an absolute part of the rows' largest possible difference
    assert torch.allclose(one.dlogits.float(), dz.float(), rtol=2.0 ** -7 if dtype == BF else 2.0 ** -12, atol=2.0 ** -12)
    ng.ngram_distill(z, t, ids, weight=weight, scale=0.5, dlogits_out=z, **kw)
    assert torch.equal(z, one.dlogits)
