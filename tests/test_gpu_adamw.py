"""ngram_adamw and ngram_adamw_rows on the GPU against the float64 step of
tests/ref8.py.

Tolerances, u = 2^-24.  fp32 results: m and v take three roundings of their
terms (4 u of the sum of absolute terms); p adds the update, whose quotient
carries about eight roundings (12 u of the quotient of m's absolute terms) and
one of p itself (3 u).
A result that is rounded at random (8-bit codes, bf16) equals the float64 one
with the same random bits, except where those errors carry the sum across a
multiple of the step: at most 16 u / 2^-4 of the codes and 16 u / 2^-8 of the
bf16 values are near enough (the chance that a uniform fraction falls within
the error of an edge), ten times that is allowed on these sizes, and then the value
is the neighbouring one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref8  # noqa: E402
from tests.ref8 import U  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32, dev, host, rounded  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
H = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1}


class Case:
    """A [rows][cols] set of parameters, gradients and moments on the host; moments in blocks along a row."""

    def __init__(self, rng, rows, cols, p_dtype, g_dtype, state):
        self.shape, self.p_dtype, self.g_dtype, self.state = (rows, cols), p_dtype, g_dtype, state
        self.p = rounded(rng.normal(size=(rows, cols)) * 0.02, p_dtype)
        self.g = rounded(rng.normal(size=(rows, cols)) * 1e-3, g_dtype)
        size = 1e-3 * np.exp(rng.normal(size=(rows, cols)))
        m, v = size * rng.normal(size=(rows, cols)) * 0.3, size * size
        if rows * cols > 40:                            # elements that never had a gradient, with and without one now
            for a in (m, v):
                a.flat[3:9] = 0.0
            self.g.flat[3:6] = 0.0
        if state == 8:
            self.m, self.ms = ref8.quant(m)
            self.v, self.vs = ref8.quant(np.sqrt(v))
        else:
            self.m, self.v = m.astype(np.float32), v.astype(np.float32)

    @property
    def nb(self):
        return ref8.ceil_div(self.shape[1], 128)

    def moments(self):
        if self.state == 32:
            return self.m.astype(np.float64), self.v.astype(np.float64)
        c = self.shape[1]
        return ref8.values(self.m, self.ms, c), ref8.values(self.v, self.vs, c) ** 2

    def device(self):
        """(p, g, m, v, m_scale, v_scale) as the calls take them."""
        t = [dev(self.p, self.p_dtype), dev(self.g, self.g_dtype)]
        if self.state == 32:
            return t + [dev(self.m), dev(self.v), None, None]
        c = self.shape[1]
        return t + [dev(self.m[:, :c]), dev(self.v[:, :c]), dev(self.ms[:, :self.nb]), dev(self.vs[:, :self.nb])]

    def check(self, got, index, step, seed, h=H, scale=1.0):
        p, m, v, ms, vs = got
        m0, v0 = self.moments()
        g = self.g.astype(np.float64) * scale
        want, wm, wv = ref8.adamw(self.p.astype(np.float64), g, m0, v0, h, step)
        word = ref8.random_words(seed, step, index)
        # the update with |m'| replaced by the sum of its absolute terms, which may cancel
        parts = h["beta1"] * np.abs(m0) + (1 - h["beta1"]) * np.abs(g)
        update = h["lr"] / (1 - h["beta1"] ** step) * parts / (np.sqrt(wv / (1 - h["beta2"] ** step)) + h["eps"])
        near = 12 * U * update + 3 * U * np.abs(self.p)
        if self.p_dtype == F32:
            assert np.all(np.abs(host(p) - want) <= near)
        else:
            up = ref8.bf16_random(want, (word >> 8) & 0xFFFF)
            diff = host(p).astype(np.float64) != up
            assert diff.mean() <= max(10 * 16 * U * 2.0 ** 8, 1.0 / diff.size)
            assert np.all(np.abs(host(p) - want) <= 2 * ref8.bf16_half_step(want) * (1 + 2.0 ** -7) + near)
        if self.state == 32:
            assert np.all(np.abs(host(m) - wm) <= 4 * U * (np.abs(0.9 * m0) + np.abs(0.1 * g)) + 1e-44)
            assert np.all(np.abs(host(v) - wv) <= 5 * U * wv + 1e-44)
            return
        c = self.shape[1]
        for codes, scales, x, w, positive in ((m, ms, wm, word & 0xFFFFF, False), (v, vs, np.sqrt(wv), word >> 12, True)):
            pad = lambda a: ref8.padded(a.astype(np.float64))  # noqa: E731
            wc, wscale, _ = ref8.pack_state(pad(x), pad(w).astype(np.int64), positive)
            codes, scales = codes.view(torch.uint8).cpu().numpy().reshape(self.shape), scales.cpu().numpy().reshape(-1, self.nb)
            bad = scales != wscale
            assert bad.mean() <= 1e-3
            # compared as numbers: where m cancels to about nothing its sign is nobody's
            diff = (ref8.decode(codes) != ref8.decode(wc[:, :c])) & ~np.repeat(bad, 128, axis=1)[:, :c]
            assert diff.mean() <= max(10 * 16 * U * 2.0 ** 4, 1.0 / diff.size)
            unit = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 128, axis=1)[:, :c]
            val = ref8.decode(codes) * unit
            gap = ref8.step_at(np.abs(x) * (1 + 8 * U) / unit) * unit
            assert np.all(np.abs(val - x) <= gap * (1 + 2.0 ** -18))
            if positive:
                assert np.all((val > 0) == (x > 0))


KINDS = [(p, g, s) for p in (BF, F32) for g in (BF, F32) for s in (8, 32)]


@pytest.mark.parametrize("p_dtype,g_dtype,state", KINDS)
def test_many_tensors(p_dtype, g_dtype, state):
    say(f"adamw {p_dtype} {g_dtype} {state}")
    rng = np.random.default_rng(1)
    sizes = [1, 7, 8, 127, 128, 129, 2047, 2560, 8191, 8192, 8193, 20_001, 0] + [300 + i for i in range(60)]
    cases = [Case(rng, 1, n, p_dtype, g_dtype, state) for n in sizes if n]
    cases.insert(5, None)                               # a tensor without elements
    parts = [c.device() if c else [torch.empty(0, dtype=p_dtype, device=DEV), torch.empty(0, dtype=g_dtype, device=DEV)]
             + ([torch.empty(0, device=DEV)] * 2 + [None] * 2 if state == 32 else [torch.empty(0, dtype=torch.uint8, device=DEV)] * 4)
             for c in cases]
    offsets = [8 * (i * 4096 + (1 << 33 if i % 2 else 0)) for i in range(len(cases))]
    lists = list(zip(*parts))
    t = ng.AdamWTensors(*lists[:4], m_scales=lists[4] if state == 8 else None, v_scales=lists[5] if state == 8 else None,
                        rng_offsets=offsets)
    ng.ngram_adamw(t, step=7, seed=123, grad_scale=0.5, **H)
    for c, x, o in zip(cases, parts, offsets):
        if c:
            n = c.shape[1]
            c.check((x[0], x[2], x[3], x[4], x[5]), (o + np.arange(n))[None], 7, 123, scale=0.5)


def test_mixed_kinds_in_one_call_and_first_step():
    say("mixed kinds, step 1")
    rng = np.random.default_rng(2)
    cases = [Case(rng, 1, 1000 + i, *k) for i, k in enumerate(KINDS)]
    parts = [c.device() for c in cases]
    lists = list(zip(*parts))
    t = ng.AdamWTensors(*lists[:4], m_scales=lists[4], v_scales=lists[5])
    ng.ngram_adamw(t, step=1, seed=(1 << 64) - 1, **H)
    at = 0
    for c, x in zip(cases, parts):
        n = c.shape[1]
        c.check((x[0], x[2], x[3], x[4], x[5]), (at + np.arange(n))[None], 1, (1 << 64) - 1)
        at += ref8.ceil_div(n, 128) * 128


@pytest.mark.parametrize("p_dtype,g_dtype,state", KINDS)
@pytest.mark.parametrize("d", [8, 136, 520, 2560])
def test_rows(p_dtype, g_dtype, state, d):
    say(f"adamw_rows d={d} {p_dtype} {g_dtype} {state}")
    rng = np.random.default_rng(d)
    R, U_rows, room = 90, 37, 50
    c = Case(rng, R, d, p_dtype, g_dtype, state)
    rows = np.sort(rng.permutation(R)[:room]).astype(np.int32)
    rows[4], rows[5] = -1, R                            # skipped
    p, _, m, v, ms, vs = c.device()
    before = [t.clone() for t in (p, m, v)]
    g = np.zeros((room, d), np.float32)
    for u in range(room):
        g[u] = c.g[rows[u]] if 0 <= rows[u] < R else 1.0
    ng.ngram_adamw_rows(p, m, v, dev(rows), dev(g, g_dtype), torch.tensor([U_rows], device=DEV), m_scale=ms, v_scale=vs, step=3,
                        seed=5, **H)
    hit = [r for r in rows[:U_rows] if 0 <= r < R]
    sub = Case.__new__(Case)
    sub.__dict__.update(c.__dict__)
    sub.shape, sub.p, sub.g = (len(hit), d), c.p[hit], c.g[hit]
    sub.m, sub.v = c.m[hit], c.v[hit]
    if state == 8:
        sub.ms, sub.vs = c.ms[hit], c.vs[hit]
    take = lambda t: None if t is None else t[torch.tensor(hit, device=DEV)]  # noqa: E731
    index = np.array(hit, dtype=np.int64)[:, None] * d + np.arange(d)
    sub.check((take(p), take(m), take(v), take(ms), take(vs)), index, 3, 5)
    rest = torch.tensor([r for r in range(R) if r not in hit], device=DEV)
    for a, b in zip((p, m, v), before):
        assert torch.equal(a[rest], b[rest])


def test_rows_from_the_table_gradient():
    """ngram_grad_table's outputs go straight in: the same bits as the step on the gathered rows."""
    say("rows from ngram_grad_table")
    rng = np.random.default_rng(8)
    n, d, R = 300, 264, 5000
    rows = torch.from_numpy(rng.integers(0, 900, (n, 16)).astype(np.int32)).to(DEV)
    dout, W = dev(rng.normal(size=(n, d)) * 1e-3, BF), dev(np.ones(d, np.float32))
    ids, grad, count = ng.ngram_grad_table(rows, W, dout, R)
    c = Case(rng, R, d, BF, F32, 8)
    p, _, m, v, ms, vs = c.device()
    ng.ngram_adamw_rows(p, m, v, ids, grad, count, m_scale=ms, v_scale=vs, step=2, seed=1, **H)
    q, _, m2, v2, ms2, vs2 = c.device()
    k = int(count.item())
    assert 100 < k <= 900
    ng.ngram_adamw_rows(q, m2, v2, ids[:k].contiguous(), grad[:k].contiguous(), m_scale=ms2, v_scale=vs2, step=2, seed=1, **H)
    for a, b in ((p, q), (m, m2), (v, v2), (ms, ms2), (vs, vs2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("state", [8, 32])
def test_not_finite_gradients_stay_where_they_are(state):
    say(f"infinite and NaN gradients {state}")
    rng = np.random.default_rng(3)
    c = Case(rng, 1, 640, BF, F32, state)
    p, g, m, v, ms, vs = c.device()
    g.view(-1)[[10, 300]] = torch.tensor([float("inf"), float("nan")], device=DEV)
    one = lambda t: None if t is None else [t]  # noqa: E731
    ng.ngram_adamw(ng.AdamWTensors([p], [g], [m], [v], one(ms), one(vs)), step=3, **H)
    bad = torch.zeros(640, dtype=torch.bool, device=DEV)
    bad[[10, 300]] = True
    got = torch.isnan(p.view(-1).float())
    assert torch.equal(got[300:301], bad[300:301]) and not torch.any(got & ~bad)
    if state == 8:
        mc = m.view(-1).view(torch.uint8)
        assert torch.equal((mc & 0x7F) == 0x7F, bad)
        assert torch.all(ms.view(-1) < 150)             # the block's scale follows its finite values


def test_a_small_second_moment_never_becomes_zero():
    say("sqrt(v) stays positive")
    n = 1024
    g = torch.full((n,), 1e-9, device=DEV)
    g[::128] = 1.0                                      # 2^-30 of the block's largest: below the smallest code
    p = torch.zeros(n, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.full((n // 128,), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    t = ng.AdamWTensors([p], [g], [m], [v], [ms], [vs])
    for step in range(1, 6):
        ng.ngram_adamw(t, step=step, seed=3, **H)
        assert torch.all(v > 0) and torch.all(v < 0x7F)
        assert torch.isfinite(p).all()


def test_equal_inputs_equal_bits_other_seed_other_bits():
    say("reproducible")
    rng = np.random.default_rng(4)
    c = Case(rng, 1, 5000, BF, BF, 8)

    def once(seed, step=2):
        x = c.device()
        ng.ngram_adamw(ng.AdamWTensors([x[0]], [x[1]], [x[2]], [x[3]], [x[4]], [x[5]]), step=step, seed=seed, **H)
        return torch.cat([x[0].view(torch.uint8).view(-1), x[2].view(-1), x[3].view(-1)])

    a = once(1)
    assert torch.equal(a, once(1)) and not torch.equal(a, once(2)) and not torch.equal(once(1, 5), once(1, 6))


def test_graph_replays():
    say("graph")
    rng = np.random.default_rng(6)
    c, r = Case(rng, 1, 9000, BF, F32, 8), Case(rng, 40, 264, BF, F32, 8)
    x, y = c.device(), r.device()
    rows = dev(np.arange(0, 40, 3).astype(np.int32))
    g = y[1][rows.long()].contiguous()
    t = ng.AdamWTensors([x[0]], [x[1]], [x[2]], [x[3]], [x[4]], [x[5]])
    state = [x[0], x[2], x[3], x[4], x[5], y[0], y[2], y[3], y[4], y[5]]
    first = [s.clone() for s in state]

    def work():
        ng.ngram_adamw(t, step=2, seed=1, **H)
        ng.ngram_adamw_rows(y[0], y[2], y[3], rows, g, m_scale=y[4], v_scale=y[5], step=2, seed=1, **H)

    def reset():
        for s, f in zip(state, first):
            s.copy_(f)
        torch.cuda.synchronize()

    work()
    torch.cuda.synchronize()
    want = [s.clone() for s in state]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        work()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            work()
    for _ in range(4):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, w) for s, w in zip(state, want))


def test_refusals():
    say("refusals of the binding")
    p, g = torch.zeros(64, device=DEV), torch.zeros(64, device=DEV)
    m, v = torch.zeros(64, device=DEV), torch.zeros(64, device=DEV)
    c8, s8 = torch.zeros(64, dtype=torch.uint8, device=DEV), torch.zeros(1, dtype=torch.uint8, device=DEV)
    ok = ng.AdamWTensors([p], [g], [m], [v])
    bad = [
        lambda: ng.AdamWTensors([p.cpu()], [g], [m], [v]),
        lambda: ng.AdamWTensors([p.half()], [g], [m], [v]),
        lambda: ng.AdamWTensors([p], [g[:32]], [m], [v]),
        lambda: ng.AdamWTensors([p], [g], [m[:8]], [v]),
        lambda: ng.AdamWTensors([p], [g], [c8], [c8]),
        lambda: ng.AdamWTensors([p], [g], [m], [v], [s8], [s8]),
        lambda: ng.AdamWTensors([p, p], [g], [m], [v]),
        lambda: ng.ngram_adamw(ok, lr=1e-3, step=0),
        lambda: ng.ngram_adamw(ok, lr=float("nan"), step=1),
        lambda: ng.ngram_adamw(ok, lr=1e-3, step=1, beta1=1.0),
        lambda: ng.ngram_adamw(ok, lr=1e-3, step=1, eps=0.0),
        lambda: ng.ngram_adamw(ng.AdamWTensors([p], [g], [m], [v], rng_offsets=[4]), lr=1e-3, step=1),
        lambda: ng.ngram_adamw(ng.AdamWTensors([p[1:]], [g[1:]], [m[1:]], [v[1:]]), lr=1e-3, step=1),
        lambda: ng.ngram_adamw_rows(p, m, v, torch.zeros(1, dtype=torch.int32, device=DEV), g, lr=1e-3, step=1),
        lambda: ng.ngram_adamw_rows(p.view(8, 8), m, v, torch.zeros(9, dtype=torch.int32, device=DEV), g, lr=1e-3, step=1),
        lambda: ng.ngram_adamw_rows(p.view(4, 16)[:, :12].contiguous(), m, v, torch.zeros(1, dtype=torch.int32, device=DEV), g, lr=1e-3, step=1),
    ]
    for f in bad:
        with pytest.raises(ng.NgramError):
            f()
    assert torch.all(p == 0)
