"""A caller's workspace that a kernel could not write is turned away before the
library sees its address.  No GPU: the library is a stand-in that must not be
called to launch."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402


class Library:
    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096

        def call(*a):
            raise AssertionError(f"{name} was called")
        return call


class OnDevice:
    """A tensor's face: on the device, of 2^20 bytes, contiguous or expanded from one element."""

    def __init__(self, contiguous):
        self.dtype, self.is_cuda, self._c = torch.uint8, True, contiguous

    def is_contiguous(self):
        return self._c

    def numel(self):
        return 1 << 20

    def element_size(self):
        return 1

    def data_ptr(self):
        return 0x10000


@pytest.mark.parametrize("workspace", [torch.empty(1 << 20, dtype=torch.uint8), OnDevice(False)], ids=["host", "expanded"])
def test_refused(workspace, monkeypatch):
    monkeypatch.setattr(ng, "lib", Library)
    monkeypatch.setattr(ng, "_arg", lambda t, *a: 0x10000)
    monkeypatch.setattr(ng, "_raw_stream", lambda s: 0)
    x, r, g = torch.zeros((4, 64)), torch.zeros(4), torch.zeros(64)
    with pytest.raises(ng.NgramError, match="workspace"):
        ng.ngram_add_norm_grad(x, x, r, g, dx_out=x, dgamma_out=g, workspace=workspace)
    q = ng.Fp8.__new__(ng.Fp8)
    q.rows, q.cols, q.block_rows, q.codes, q.scales, q.c = 64, 128, 1, x, x, None
    with pytest.raises(ng.NgramError, match="workspace"):
        ng.ngram_project_fp8(q, q, out=x, workspace=workspace)


def test_taken(monkeypatch):
    """A contiguous device tensor reaches the library with its bytes."""
    class Takes(Library):
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 4096
            return lambda *a: 0 if 0x10000 in a and (1 << 20) in a else -1
    monkeypatch.setattr(ng, "lib", Takes)
    monkeypatch.setattr(ng, "_arg", lambda t, *a: 1)
    monkeypatch.setattr(ng, "_raw_stream", lambda s: 0)
    monkeypatch.setattr(ng, "_check", lambda rc, what: 1 / 0)
    x, r, g = torch.zeros((4, 64)), torch.zeros(4), torch.zeros(64)
    ng.ngram_add_norm_grad(x, x, r, g, dx_out=x, dgamma_out=g, workspace=OnDevice(True))


def test_no_8_bit_matrix_in_host_memory(monkeypatch):
    """Fp8.empty of a device that kernels cannot write."""
    for device in ("cpu", torch.device("cpu"), "meta"):
        with pytest.raises(ng.NgramError, match="device"):
            ng.Fp8.empty(4, 64, device=device)
