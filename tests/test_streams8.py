"""Where the 8-bit calls' own tensors come from: memory that a call makes for a
given stream is taken on that stream, so that it is never a block which work
queued on the current stream still uses.  No GPU: the allocator, the streams and
the library are stand-ins that write down what happens."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402


class Stream:
    def __init__(self, name):
        self.name, self.cuda_stream = name, 0


class Library:
    """Takes every call; workspaces are 4096 bytes."""

    def __getattr__(self, name):
        return (lambda *a: 4096) if name.endswith("workspace_bytes") else (lambda *a: 0)


@pytest.fixture
def made(monkeypatch):
    """What is allocated, as (stream at the time, streams recorded)."""
    at, log, recorded = [Stream("current")], [], {}

    @contextlib.contextmanager
    def on(stream):
        at.append(stream)
        yield
        at.pop()

    def allocator(real):
        def take(*a, **kw):
            kw.pop("device", None)
            t = real(*a, **kw)
            log.append((at[-1].name, t))
            return t
        return take

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: at[-1])
    monkeypatch.setattr(torch, "empty_strided", allocator(torch.empty_strided))
    monkeypatch.setattr(torch, "empty", allocator(torch.empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.setdefault(id(t), []).append(s.name))
    monkeypatch.setattr(ng, "lib", Library)
    monkeypatch.setattr(ng, "_arg", lambda t, *a: t.data_ptr())
    if hasattr(ng, "_scratch"):
        monkeypatch.setattr(ng, "_scratch", lambda t: (t.data_ptr(), t.numel()))
    return log, recorded


X = torch.zeros((5, 16))
R, G = torch.zeros(5), torch.zeros(16)
Q = ng.Fp8.__new__(ng.Fp8)
Q.rows, Q.cols, Q.block_rows, Q.codes, Q.scales, Q.c = 64, 128, 1, X, X, None

CALLS = {
    "quant": (lambda s: ng.ngram_quant_fp8(X, transposed=True, stream=s), 4),
    "norm": (lambda s: ng.ngram_add_norm(X, G, 1e-6, keep_y=True, keep_r=True, stream=s), 4),
    "norm_grad": (lambda s: ng.ngram_add_norm_grad(X, X, R, G, stream=s), 3),
    "project": (lambda s: ng.ngram_project_fp8(Q, Q, stream=s), 2),
    "fp8": (lambda s: ng.Fp8.empty(5, 16, stream=s), 2),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_a_call_are_taken_on_its_stream(name, made):
    log, recorded = made
    call, count = CALLS[name]
    call(Stream("side"))
    assert [s for s, _ in log] == ["side"] * count
    # the results are the caller's, who reads them on the current stream: the allocator is told
    results = [t for _, t in log if t.dtype != torch.uint8 or t.dim() == 2]
    assert results and all("current" in recorded.get(id(t), []) for t in results)


@pytest.mark.parametrize("name", [n for n in CALLS if n != "fp8"])
def test_without_a_stream_the_current_one_is_used(name, made, monkeypatch):
    monkeypatch.setattr(ng, "_raw_stream", lambda s: 0 if s is None else 1 / 0)
    log, recorded = made
    call, count = CALLS[name]
    call(None)
    assert [s for s, _ in log] == ["current"] * count and not recorded
