"""Every tile shape of ngram_project_fp8, over one, few and many steps of 128
columns, in one item a workgroup and in several that follow each other, with K
whole and split, and ragged in both directions: the whole result against a
float64 product.

Tolerances, as in test_gpu_product_bits.py: fp32 sums of exact products, 2 (K +
8) u of the sum of absolute terms; the 8-bit instruction cuts each group of
eight columns by less than 2^(E - 10), E at most the sum of the two largest
exponents; a bf16 result half a step, and its error's norm is the rounding's to
1%."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.ref8 import U  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu

# (m, n, k, parts of K)
BF16 = {
    "64 x 64": [(100, 136, 128, 1), (136, 264, 392, 1), (264, 136, 2568, 1), (100, 136, 8200, 5), (2000, 136, 8200, 2)],
    "128 x 128": [(1000, 1032, 128, 1), (777, 2000, 392, 1), (1000, 1032, 2568, 1), (520, 2552, 8200, 2), (1000, 1032, 8200, 3),
                  (2000, 136, 16392, 7)],
    "256 x 256": [(2000, 4104, 128, 1), (1000, 8200, 392, 1), (2000, 4104, 1032, 1), (4100, 5000, 392, 1), (4100, 5000, 1160, 1),
                  (5000, 4104, 2568, 1), (1000, 4104, 8200, 3), (136, 8200, 16392, 7)],
    "256 x 320": [(4100, 4104, 128, 1), (2000, 8200, 392, 1), (4100, 4104, 1032, 1), (8200, 4104, 392, 1), (4100, 8200, 1160, 1),
                  (1000, 8200, 16392, 2), (520, 8200, 16392, 3)],
}
FP32 = {
    "64 x 64": [(100, 136, 128, 1), (136, 264, 392, 1), (264, 136, 2568, 1), (100, 136, 4232, 2), (100, 136, 8200, 5)],
    "128 x 128": [(1000, 1032, 128, 1), (777, 2000, 392, 1), (777, 2552, 2568, 1), (520, 2552, 8200, 2), (1000, 1032, 8200, 3)],
    "256 x 128": [(1000, 4104, 128, 1), (4100, 1032, 392, 1), (1000, 4104, 1032, 1), (3001, 4104, 392, 1), (2552, 5000, 1160, 1),
                  (3001, 4104, 2568, 1), (2000, 1032, 8200, 3), (4100, 264, 16392, 5)],
}
CASES = [(BF, tile, *c) for tile, cs in BF16.items() for c in cs] + [(F32, tile, *c) for tile, cs in FP32.items() for c in cs]


def matrix(g, rows, k, block_rows=1):
    x = torch.randn((rows, k), generator=g, device=DEV) * torch.exp(torch.randn((rows, 1), generator=g, device=DEV))
    wide = torch.nn.functional.pad(x * torch.exp(torch.randn((1, k), generator=g, device=DEV)), (0, -k % 8))
    return ng.ngram_quant_fp8(wide, block_rows=block_rows)[0]


def pow2(e):
    """2^e in float64, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def values(q):
    """The numbers that q holds [rows][128 blocks], and the largest 2^exponent of each eight columns, both float64."""
    codes = q.codes.view(torch.uint8)
    rows, ld = codes.shape
    scale = pow2(q.scales[:, :ld // 128].int() - 127)
    if q.block_rows == 128:
        scale = scale.repeat_interleave(128, dim=0)[:rows]
    v = (q.codes.double().view(rows, -1, 128) * scale[:, :, None]).view(rows, ld)
    top = ((codes.int() >> 3) & 15).clamp(min=1).view(rows, -1, 8).amax(dim=2) - 7
    return v, (pow2(top).view(rows, -1, 16) * scale[:, :, None]).view(rows, -1)


@pytest.mark.parametrize("dtype,tile,m,n,k,parts", CASES)
def test_tile(dtype, tile, m, n, k, parts):
    say(f"{tile} tiles, {m} x {n} x {k}, K in {parts}, {dtype}")
    workspace = ng.project_fp8_workspace(m, n, k, dtype)
    assert parts == (1 if workspace is None else workspace.numel() // (4 * m * n))
    g = torch.Generator(device=DEV).manual_seed(m + 3 * n + 7 * k)
    k8 = k + -k % 8
    a, b = matrix(g, m, k8), matrix(g, n, k8, 128 if m % 2 else 1)
    got = ng.ngram_project_fp8(a, b, dtype=dtype)
    again = ng.ngram_project_fp8(a, b, out=torch.full((m, n), float("nan"), dtype=dtype, device=DEV))
    assert torch.equal(got.view(torch.uint8), again.view(torch.uint8))
    (av, ag), (bv, bg) = values(a), values(b)
    bt = bv.t().contiguous()
    want, room = av @ bt, (av.abs() @ bt.abs()).mul_(2 * (k8 + 8) * U)
    err = (got.double() - want).abs_()
    if dtype == F32:
        assert torch.linalg.norm(err) <= 1e-6 * torch.linalg.norm(want)
    else:
        room += (ag @ bg.t().contiguous()).mul_(2.0 ** -10)
        exponent = torch.frexp(want.abs())[1].clamp(min=-125)
        room += (1 + 2.0 ** -6) * pow2(exponent - 9)
        rounding = torch.linalg.norm(want.to(BF).double() - want)
        print(f"[norm of the error] {float(torch.linalg.norm(err) / torch.linalg.norm(want)):.6f}, of the rounding alone "
              f"{float(rounding / torch.linalg.norm(want)):.6f}", flush=True)
        assert torch.linalg.norm(err) <= 1.01 * rounding
    worst = float((err / room.clamp(min=1e-300)).max())
    print(f"[error over bound] {worst:.3f}", flush=True)
    assert worst <= 1.0
