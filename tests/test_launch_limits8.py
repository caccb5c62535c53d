"""Sizes of the 8-bit calls that no launch covers are turned away on the host
before anything is launched.  No GPU."""
import ctypes

import pytest

import hashed_gram_embedding_ngram_amd as ng

ERANGE = -3
A = 0x10000             # a fake, aligned device address (never dereferenced)


def fp8(rows, cols, block_rows=1):
    return ctypes.byref(ng._Fp8(A, A, rows, cols, block_rows, 0))


@pytest.mark.parametrize("n,d", [(1 << 30, 136), (1 << 30, 65536), (1 << 23, 65536)])
def test_quantiser_of_too_many_tiles(n, d):
    """A workgroup of 256 threads for a tile of 128 x 128: 2^24 - 1 tiles at most."""
    assert ng.lib().ngram_quant_fp8(A, 1, n, d, fp8(n, d), None, None) == ERANGE, ng.lib().ngram_last_error()
    assert b"too large" in ng.lib().ngram_last_error()


@pytest.mark.parametrize("m,n,dtype", [(1 << 30, 8192, 1), (1 << 30, 1 << 20, 0), (1 << 26, 1 << 26, 1)])
def test_product_of_too_many_tiles(m, n, dtype):
    """Over one step of K a workgroup has one of the large tiles; their number is a launch's limit."""
    assert ng.lib().ngram_project_fp8_workspace_bytes(m, n, 128, dtype) == 0
    assert ng.lib().ngram_project_fp8(fp8(m, 128), fp8(n, 128), A, dtype, None, 0, None) == ERANGE, ng.lib().ngram_last_error()
    assert b"too large" in ng.lib().ngram_last_error()
