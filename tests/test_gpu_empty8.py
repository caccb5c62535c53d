"""A product over no columns: the weight gradient of an empty batch is zero."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
def test_empty_batch(dtype):
    say(f"weight gradient of no rows {dtype}")
    d_in, d_out = 264, 136
    _, gt = ng.ngram_quant_fp8(torch.empty((0, d_out), dtype=BF, device=DEV), rows=False, transposed=True)
    _, xt = ng.ngram_quant_fp8(torch.empty((0, d_in), dtype=BF, device=DEV), rows=False, transposed=True)
    old = torch.full((d_out * d_in + 8,), 7.0, dtype=dtype, device=DEV)
    out = ng.ngram_project_fp8(gt, xt, out=old)
    assert torch.all(out[:d_out * d_in] == 0) and torch.all(out[d_out * d_in:] == 7.0)
    made = ng.ngram_project_fp8(gt, xt, dtype=dtype)
    assert made.shape == (d_out, d_in) and made.dtype == dtype and torch.all(made == 0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    side = ng.ngram_project_fp8(gt, xt, dtype=dtype, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.all(side == 0)
    with pytest.raises(ng.NgramError):
        ng.ngram_project_fp8(gt, ng.Fp8.empty(12, 0))           # B's rows are no multiple of 8
    with pytest.raises(ng.NgramError):
        ng.ngram_project_fp8(gt, ng.Fp8.empty(16, 128))         # other columns
    with pytest.raises(ng.NgramError):
        ng.ngram_project_fp8(gt, xt, out=old[:100])
