"""The 8-bit calls with ``stream=`` and tensors of their own making, while the
current stream still has work queued on blocks that Python has let go: the
results are those of the calls on the current stream."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, F32, dev  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 1e-6


def busy(sizes):
    """Queue some milliseconds of work on the current stream, then stores to blocks of these sizes, which are let go at once."""
    a = torch.zeros((4096, 4096), device=DEV)
    blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    for _ in range(20):
        a = a @ a
    for b in blocks:
        b.fill_(0x55)


def test_results_while_the_current_stream_is_busy():
    say("stream= beside a busy current stream")
    rng = np.random.default_rng(4)
    n, d, o = 700, 2560, 264
    x, dy = dev(rng.normal(size=(n, d)), BF), dev(rng.normal(size=(n, d)), F32)
    gamma = torch.ones(d, device=DEV)
    P, _ = ng.ngram_quant_fp8(dev(rng.normal(size=(o, d)), F32))
    long = [ng.ngram_quant_fp8(dev(rng.normal(size=(136, 16392)), F32))[0] for _ in range(2)]
    assert ng.project_fp8_workspace(136, 136, 16392) is not None
    total = torch.empty((n, d), dtype=BF, device=DEV)

    def work(stream):
        norm = ng.ngram_add_norm(x, gamma, EPS, sum_out=total, keep_y=True, keep_r=True, stream=stream)
        dx, dg = ng.ngram_add_norm_grad(dy, total, norm.r, gamma, stream=stream)
        q, qt = ng.ngram_quant_fp8(dx, transposed=True, stream=stream)
        y = ng.ngram_project_fp8(norm.q, P, stream=stream)
        z = ng.ngram_project_fp8(*long, dtype=F32, stream=stream)
        return [total, norm.y, norm.r, norm.q.codes, norm.q.scales, dx, dg, q.codes, q.scales, qt.codes, qt.scales, y, z]

    want = [t.clone() for t in work(None)]
    sizes = sorted({t.numel() * t.element_size() for t in want} | {ng.add_norm_grad_workspace(n, d).numel(),
                                                                   ng.project_fp8_workspace(136, 136, 16392).numel()})
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy(sizes)
        got = work(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def test_results_let_go_while_they_are_read():
    """A result read on the current stream after its last reference is gone: a later call on the side stream leaves it."""
    say("results of a side stream read late")
    rng = np.random.default_rng(5)
    a, b = (ng.ngram_quant_fp8(dev(rng.normal(size=(512, 256)), F32))[0] for _ in range(2))
    c, _ = ng.ngram_quant_fp8(torch.zeros((512, 256), device=DEV))
    want = ng.ngram_project_fp8(a, b, dtype=F32).clone()
    side, seen = torch.cuda.Stream(), torch.empty_like(want)
    m = torch.zeros((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        out = ng.ngram_project_fp8(a, b, dtype=F32, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(20):
            m = m @ m
        seen.copy_(out)
        del out
        for _ in range(4):
            ng.ngram_project_fp8(c, b, dtype=F32, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(seen, want)
