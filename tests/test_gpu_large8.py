"""The 8-bit operators where element offsets pass 2^31: the last rows of a
large call equal a small call on copies of those rows, bit for bit."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def u8(t):
    return t.view(torch.uint8)


def test_norm_and_quantiser_beyond_2_31():
    n, d = 850_000, 2560
    assert n * d > 1 << 31
    say(f"norm {n} x {d}")
    x = torch.empty((n, d), dtype=BF, device=DEV).normal_()
    gamma = torch.rand(d, device=DEV)
    last = slice(n - 2100, n)
    out = ng.ngram_add_norm(x, gamma, 1e-6, keep_r=True)
    small = ng.ngram_add_norm(x[last].contiguous(), gamma, 1e-6, keep_r=True)
    assert torch.equal(u8(out.q.codes[last]), u8(small.q.codes)) and torch.equal(out.q.scales[last], small.q.scales)
    assert torch.equal(out.r[last], small.r)
    dx, _ = ng.ngram_add_norm_grad(x, x, out.r, gamma)
    few, _ = ng.ngram_add_norm_grad(x[last].contiguous(), x[last].contiguous(), small.r, gamma)
    assert torch.equal(dx[last], few)
    del dx, out
    q, qt = ng.ngram_quant_fp8(x, transposed=True)
    cut = n // 128 * 128 - 128
    sq, st = ng.ngram_quant_fp8(x[cut:].contiguous(), transposed=True)
    assert torch.equal(u8(q.codes[cut:]), u8(sq.codes)) and torch.equal(u8(qt.codes[:, cut:]), u8(st.codes))
    assert torch.equal(qt.scales[:, cut // 128:cut // 128 + 2], st.scales[:, :2])


def test_product_result_beyond_2_31():
    m, n, k = 1_100_000, 2560, 256
    assert m * n > 1 << 31
    say(f"product {m} x {n} x {k}")
    a = ng.ngram_quant_fp8(torch.randn(m, k, device=DEV))[0]
    b = ng.ngram_quant_fp8(torch.randn(n, k, device=DEV))[0]
    big = ng.ngram_project_fp8(a, b)
    at = m - 5000
    small = ng.ngram_project_fp8(ng.Fp8(a.codes[at:].contiguous(), a.scales[at:].contiguous(), 5000, k), b)
    # the two calls may take different tiles, hence sums in another order: bf16 neighbours at most
    x, y = big[at:].float(), small.float()
    assert torch.all((x - y).abs() <= 2.0 ** -7 * y.abs() + 1e-2) and torch.linalg.norm(x - y) <= 1e-3 * torch.linalg.norm(y)


def test_rows_of_a_table_beyond_2_31():
    R, d = 900_000, 2560
    assert R * d > 1 << 31
    say(f"adamw_rows on {R} x {d}")
    p = torch.empty((R, d), dtype=BF, device=DEV).normal_(std=0.02)
    m, v = (torch.zeros((R, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.full((R, d // 128), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    rows = torch.tensor([0, 5, R - 3, R - 1], dtype=torch.int32, device=DEV)
    g = torch.randn((4, d), device=DEV)
    before = p[rows.long()].clone()
    ng.ngram_adamw_rows(p, m, v, rows, g, m_scale=ms, v_scale=vs, lr=1e-2, step=1)
    # the first step moves each parameter by lr against its gradient's sign, to within a bf16 step and the weight decay
    moved = p[rows.long()].float() - before.float()
    assert torch.all((moved + 1e-2 * g.sign()).abs() <= 2.0 ** -7 * (before.float().abs() + 1e-2) + 1e-6)
    for t in (m, v):
        hit = t.view(R, d)[rows.long()]
        assert torch.all(hit[:, :] != 0) or (hit != 0).float().mean() > 0.99
        assert int((t.view(torch.int64) != 0).any(dim=1).sum()) == 4


def test_a_tensor_beyond_2_31():
    n = (1 << 31) + 4096 + 24
    say(f"adamw on {n} elements")
    p = torch.zeros(n, dtype=BF, device=DEV)
    g = torch.ones(n, dtype=BF, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.full((-(-n // 128),), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    ng.ngram_adamw(ng.AdamWTensors([p], [g], [m], [v], [ms], [vs]), lr=1e-2, step=1)
    tail = p[-5000:].float()
    assert torch.all((tail + 1e-2).abs() <= 1e-4) and torch.all(m[-5000:] != 0) and torch.all(v[-5000:] != 0)
    assert torch.all((p[:5000].float() + 1e-2).abs() <= 1e-4)
