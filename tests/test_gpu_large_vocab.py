"""The vocabulary's operators where offsets pass 2^31 and 2^32: rows at the end
equal a call on copies of those rows, bit for bit."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def test_4_bit_matrix_beyond_2_31():
    rows, cols = 1_700_000, 2560
    assert rows * cols // 2 > 1 << 31
    say(f"4-bit {rows} x {cols}")
    x = torch.empty((rows, cols), dtype=BF, device=DEV).normal_()
    last = slice(rows - 2100, rows)
    q, small = ng.ngram_quant_int4(x, 64), ng.ngram_quant_int4(x[last].contiguous(), 64)
    for a, b in ((q.codes, small.codes), (q.scales, small.scales), (q.zeros, small.zeros)):
        assert torch.equal(a.view(rows, -1)[last], b.view(2100, -1))
    x3 = torch.randn((3, cols), device=DEV).to(BF)
    assert torch.equal(ng.ngram_project_int4(x3, q)[:, last], ng.ngram_project_int4(x3, small))
    y = ng.ngram_dequant_int4(q, out=x)
    assert torch.equal(y[last], ng.ngram_dequant_int4(small, dtype=BF))


def test_product_result_beyond_2_31():
    """Whole numbers, whose sums are exact in any order."""
    n, cols, rows = 1300, 264, 1_700_000
    assert n * rows > 1 << 31
    say(f"4-bit product {n} x {cols} x {rows}")
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randint(-3, 4, (n, cols), generator=g, device=DEV).to(BF)
    codes = torch.randint(0, 256, (rows, 144), generator=g, device=DEV).to(torch.uint8)
    scales = torch.ones((rows, 4), dtype=BF, device=DEV)
    y = ng.ngram_project_int4(x, ng.Int4(codes, scales, rows, cols), dtype=F32)
    at = rows - 300
    small = ng.ngram_project_int4(x, ng.Int4(codes[at:].contiguous(), scales[at:].contiguous(), 300, cols), dtype=F32)
    assert torch.equal(y[:, at:], small)
    values = ng.ngram_dequant_int4(ng.Int4(codes[at:].contiguous(), scales[at:].contiguous(), 300, cols)).cpu().double()
    assert torch.equal(small.cpu().double(), x.cpu().double() @ values.t())


@pytest.mark.parametrize("V", [5003, 70001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_logits_beyond_2_31(V, dtype):
    n, ld, k = 3, (1 << 30) + 9, 40
    assert (n - 1) * ld > 1 << 31
    say(f"logits {n} x {V}, {ld} apart, {dtype}")
    g = torch.Generator(device=DEV).manual_seed(V)
    far, dfar = (torch.empty((n - 1) * ld + V, dtype=dtype, device=DEV).as_strided((n, V), (ld, 1)) for _ in range(2))
    z = torch.randn((n, V), generator=g, device=DEV).to(dtype)
    far.copy_(z)
    scores = torch.tensor([-1.0, -0.5, -2.0], device=DEV)
    for a, b in zip(ng.ngram_beam_step(far, scores, n, end_token=3), ng.ngram_beam_step(z, scores, n, end_token=3)):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    t = torch.randn((n, k), generator=g, device=DEV)
    ids = torch.randint(0, V, (n, k), generator=g, device=DEV).int()
    ids[:, 0] = V - 1
    want = ng.ngram_distill(z, t, ids, 1.5, grad=True, keep_stats=True)
    got = ng.ngram_distill(far, t, ids, 1.5, keep_stats=True, dlogits_out=dfar)
    assert torch.equal(got.loss, want.loss) and torch.equal(got.stats, want.stats) and torch.equal(dfar, want.dlogits)
    dfar.zero_()
    ng.ngram_distill_grad(far, t, ids, got.stats, 1.5, dlogits_out=dfar)
    assert torch.equal(dfar, ng.ngram_distill_grad(z, t, ids, want.stats, 1.5))


def test_states_beyond_2_32():
    say("reorder far rows and long ones")
    far = torch.empty(3 * ((1 << 31) + 16) + 48, dtype=torch.uint8, device=DEV).as_strided((4, 48), ((1 << 31) + 16, 1))
    far.copy_(torch.arange(192, device=DEV).view(4, 48))
    long = torch.zeros((4, (1 << 32) + 4112), dtype=torch.uint8, device=DEV)
    for b in range(4):
        long[b, :4112] = b + 1
        long[b, -4112:] = 11 * (b + 1)
    parents = torch.tensor([1, 0, 3, 1], dtype=torch.int32, device=DEV)
    want = far[parents.long()].clone()
    ng.ngram_beam_reorder(ng.BeamStates([far, long]), parents, 4)
    assert torch.equal(far, want)
    for b, p in enumerate([1, 0, 3, 1]):
        assert torch.all(long[b, :4112] == p + 1) and torch.all(long[b, -4112:] == 11 * (p + 1))
        assert torch.all(long[b, (1 << 31):(1 << 31) + 4096] == 0)
