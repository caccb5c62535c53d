"""Workspaces that the 8-bit calls refuse on the device: nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_refusals():
    say("workspaces that are refused")
    n, d = 1500, 136
    x, r, g = torch.zeros((n, d), dtype=torch.bfloat16, device=DEV), torch.ones(n, device=DEV), torch.ones(d, device=DEV)
    size = ng.add_norm_grad_workspace(n, d).numel()
    long = [ng.ngram_quant_fp8(torch.randn(136, 16392, device=DEV))[0] for _ in range(2)]
    split = ng.project_fp8_workspace(136, 136, 16392, torch.bfloat16).numel()
    one = torch.zeros(1, dtype=torch.uint8, device=DEV)
    bad = [lambda b: torch.empty(b, dtype=torch.uint8), lambda b: one.expand(b), lambda b: torch.empty(2 * b, dtype=torch.uint8, device=DEV)[::2]]
    dx, dg, out = torch.full_like(x, 7.0), torch.full((d,), 7.0, device=DEV), torch.full((136, 136), 7.0, device=DEV)
    for make in bad:
        with pytest.raises(ng.NgramError):
            ng.ngram_add_norm_grad(x, x, r, g, dx_out=dx, dgamma_out=dg, workspace=make(size))
        with pytest.raises(ng.NgramError):
            ng.ngram_project_fp8(*long, out=out, workspace=make(max(split, ng.project_fp8_workspace(136, 136, 16392).numel())))
    torch.cuda.synchronize()
    assert torch.all(dx == 7.0) and torch.all(dg == 7.0) and torch.all(out == 7.0) and int(one) == 0
    # a workspace of another type than bytes is taken
    ng.ngram_add_norm_grad(x, x, r, g, dx_out=dx, dgamma_out=dg, workspace=torch.empty(size // 4 + 1, device=DEV))
    assert torch.all(dx == 0) and torch.all(dg == 0)
