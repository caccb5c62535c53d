"""The 8-bit calls of the C ABI without a GPU: sizes, and bad arguments turned
away on the host with the documented status codes before anything is launched."""
import ctypes
import os
import re

import pytest

import hashed_gram_embedding_ngram_amd as ng

OK, EINVAL, EALIGN, ERANGE = 0, -1, -2, -3
A = 0x10000             # a fake, aligned device address (never dereferenced)
MAX = 1 << 30


def fp8(codes=A, scales=A, rows=16, cols=256, block_rows=1):
    return ctypes.byref(ng._Fp8(codes, scales, rows, cols, block_rows, 0))


def test_sizes():
    L = ng.lib()
    assert L.ngram_fp8_code_bytes(3, 129) == 3 * 256 and L.ngram_fp8_code_bytes(0, 5) == 0
    assert L.ngram_fp8_scale_bytes(3, 129, 1) == 3 * 4 and L.ngram_fp8_scale_bytes(129, 513, 128) == 2 * 8
    for bad in ((-1, 5), (5, -1), (MAX + 1, 5), (5, MAX + 1)):
        assert L.ngram_fp8_code_bytes(*bad) == -1 and L.ngram_fp8_scale_bytes(*bad, 1) == -1
    assert L.ngram_fp8_scale_bytes(5, 5, 64) == -1
    assert L.ngram_add_norm_grad_workspace_bytes(5, 12) == -1 and L.ngram_add_norm_grad_workspace_bytes(-1, 8) == -1
    assert L.ngram_add_norm_grad_workspace_bytes(5, 65544) == -1 and L.ngram_add_norm_grad_workspace_bytes(0, 64) > 0
    assert L.ngram_project_fp8_workspace_bytes(5, 12, 64, 0) == -1 and L.ngram_project_fp8_workspace_bytes(5, 8, (1 << 23) + 1, 0) == -1
    assert L.ngram_project_fp8_workspace_bytes(4, 2560, 2560, 1) >= 0 and L.ngram_project_fp8_workspace_bytes(4, 8, 8, 2) == -1


def norm(x=A, xt=1, res=A, n=4, d=64, gamma=A, eps=1e-6, s=A, y=A, q=None, r=None):
    return ng.lib().ngram_add_norm(x, xt, res, n, d, gamma, eps, s, y, q, r, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), EINVAL), (dict(d=0), EINVAL), (dict(d=12), EINVAL), (dict(d=65544), ERANGE), (dict(n=MAX + 1), ERANGE),
    (dict(xt=2), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("inf")), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(x=None), EINVAL), (dict(gamma=None), EINVAL), (dict(s=None, y=None), EINVAL), (dict(x=A + 8), EALIGN),
    (dict(res=A + 2), EALIGN), (dict(gamma=A + 4), EALIGN), (dict(s=A + 8), EALIGN), (dict(y=A + 8), EALIGN),
    (dict(r=A + 2), EALIGN), (dict(q=fp8(rows=4, cols=128)), EINVAL), (dict(q=fp8(rows=4, cols=64, block_rows=128)), EINVAL),
    (dict(q=fp8(codes=None, rows=4, cols=64)), EINVAL), (dict(q=fp8(codes=A + 8, rows=4, cols=64)), EALIGN),
    (dict(q=fp8(scales=A + 2, rows=4, cols=64)), EALIGN), (dict(q=fp8(rows=4, cols=64, block_rows=3)), EINVAL),
    (dict(n=0, x=None, s=None, y=None), OK),
])
def test_add_norm_refuses(kw, code):
    assert norm(**kw) == code, ng.lib().ngram_last_error()


def test_error_messages_share_one_buffer():
    L = ng.lib()
    assert norm(d=12) == EINVAL and b"d=12" in L.ngram_last_error()
    assert norm(n=0) == OK and L.ngram_last_error() == b""
    assert L.ngram_hash(A, -1, A, 1, None, None, 10, A, None) == EINVAL and b"n=-1" in L.ngram_last_error()
    with pytest.raises(ng.NgramError, match="d=12"):
        ng._check(norm(d=12), "ngram_add_norm")


def grad(dy=A, t=1, s=A, r=A, gamma=A, ds=A, n=4, d=64, dx=A, dg=A, ws=A, size=1 << 20):
    return ng.lib().ngram_add_norm_grad(dy, t, s, r, gamma, ds, n, d, dx, dg, ws, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), EINVAL), (dict(d=4), EINVAL), (dict(d=65544), ERANGE), (dict(t=-1), EINVAL), (dict(dy=None), EINVAL),
    (dict(s=None), EINVAL), (dict(r=None), EINVAL), (dict(gamma=None), EINVAL), (dict(dx=None), EINVAL), (dict(dg=None), EINVAL),
    (dict(dy=A + 8), EALIGN), (dict(s=A + 8), EALIGN), (dict(ds=A + 8), EALIGN), (dict(dx=A + 8), EALIGN), (dict(r=A + 2), EALIGN),
    (dict(ws=None), EINVAL), (dict(ws=A + 8), EINVAL), (dict(size=16), EINVAL),
])
def test_add_norm_grad_refuses(kw, code):
    assert grad(**kw) == code, ng.lib().ngram_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(q=None, qt=None), EINVAL), (dict(n=-1), EINVAL), (dict(d=12), EINVAL), (dict(t=7), EINVAL), (dict(x=None), EINVAL),
    (dict(x=A + 4), EALIGN), (dict(q=fp8(rows=16, cols=128)), EINVAL), (dict(qt=fp8(rows=16, cols=256)), EINVAL),
    (dict(qt=fp8(rows=256, cols=16, block_rows=128)), EINVAL), (dict(q=fp8(codes=A + 1)), EALIGN),
    (dict(n=0, x=None, q=fp8(rows=0), qt=fp8(rows=256, cols=0)), OK),
])
def test_quant_refuses(kw, code):
    a = dict(x=A, t=0, n=16, d=256, q=fp8(), qt=fp8(rows=256, cols=16)) | kw
    assert ng.lib().ngram_quant_fp8(a["x"], a["t"], a["n"], a["d"], a["q"], a["qt"], None) == code, ng.lib().ngram_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), EINVAL), (dict(b=None), EINVAL), (dict(t=2), EINVAL), (dict(c=None), EINVAL), (dict(c=A + 8), EALIGN),
    (dict(b=fp8(cols=128)), EINVAL), (dict(b=fp8(rows=12)), EINVAL), (dict(b=fp8(rows=0)), EINVAL), (dict(a=fp8(rows=-1)), EINVAL),
    (dict(a=fp8(cols=0), b=fp8(cols=0)), EINVAL), (dict(a=fp8(cols=(1 << 23) + 1), b=fp8(cols=(1 << 23) + 1)), ERANGE),
    (dict(a=fp8(rows=MAX + 1)), ERANGE), (dict(a=fp8(block_rows=0)), EINVAL), (dict(a=fp8(codes=None)), EINVAL),
    (dict(a=fp8(rows=136, cols=1 << 20), b=fp8(rows=136, cols=1 << 20)), EINVAL),       # K is split: a workspace is needed
    (dict(a=fp8(rows=0), c=None), OK),
])
def test_project_refuses(kw, code):
    a = dict(a=fp8(), b=fp8(), c=A, t=0) | kw
    assert ng.lib().ngram_project_fp8(a["a"], a["b"], a["c"], a["t"], None, 0, None) == code, ng.lib().ngram_last_error()


def tensor(**kw):
    f = dict(p=A, g=A, m=A, v=A, m_scale=None, v_scale=None, numel=64, rng_offset=0, p_dtype=0, g_dtype=0, state=0) | kw
    return ng._AdamWTensor(*f.values(), 0)


def step(**kw):
    f = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0, step=1, seed=0) | kw
    return ctypes.byref(ng._AdamWStep(*f.values()))


BAD_TENSORS = [
    (dict(p=None), EINVAL), (dict(g=None), EINVAL), (dict(m=None), EINVAL), (dict(v=None), EINVAL), (dict(state=1), EINVAL),
    (dict(state=1, m_scale=A), EINVAL), (dict(state=2), EINVAL), (dict(p_dtype=2), EINVAL), (dict(g_dtype=-1), EINVAL),
    (dict(p=A + 8), EALIGN), (dict(g=A + 8), EALIGN), (dict(m=A + 8), EALIGN), (dict(state=1, m_scale=A, v_scale=A, m=A + 4), EALIGN),
]
BAD_STEPS = [dict(step=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0),
             dict(eps=float("inf")), dict(lr=float("nan")), dict(weight_decay=float("inf")), dict(grad_scale=float("nan"))]


@pytest.mark.parametrize("kw,code", BAD_TENSORS + [
    (dict(numel=-1), EINVAL), (dict(rng_offset=4), EINVAL), (dict(rng_offset=-8), EINVAL), (dict(numel=1 << 44), ERANGE)])
def test_adamw_refuses_tensors(kw, code):
    two = (ng._AdamWTensor * 2)(tensor(), tensor(**kw))
    assert ng.lib().ngram_adamw(two, 2, step(), None) == code, ng.lib().ngram_last_error()
    assert b"tensor 1" in ng.lib().ngram_last_error() or b"dtype" in ng.lib().ngram_last_error() or b"state" in ng.lib().ngram_last_error()


@pytest.mark.parametrize("kw", BAD_STEPS)
def test_adamw_refuses_steps(kw):
    one = (ng._AdamWTensor * 1)(tensor())
    assert ng.lib().ngram_adamw(one, 1, step(**kw), None) == EINVAL
    assert ng.lib().ngram_adamw_rows(one, 8, 8, A, 1, None, step(**kw), None) == EINVAL


def test_adamw_of_nothing():
    L = ng.lib()
    one = (ng._AdamWTensor * 1)(tensor(numel=0, p=None, g=None, m=None, v=None))
    assert L.ngram_adamw(None, 0, step(), None) == OK and L.ngram_adamw(one, 1, step(), None) == OK
    assert L.ngram_adamw(None, 1, step(), None) == EINVAL and L.ngram_adamw(one, -1, step(), None) == EINVAL
    assert L.ngram_adamw(one, 1, None, None) == EINVAL


@pytest.mark.parametrize("kw,code", BAD_TENSORS + [(dict(numel=65), EINVAL), (dict(rng_offset=8), EINVAL)])
def test_adamw_rows_refuses_tables(kw, code):
    t = ctypes.byref(tensor(**kw))
    assert ng.lib().ngram_adamw_rows(t, 8, 8, A, 4, A, step(), None) == code, ng.lib().ngram_last_error()


def test_adamw_rows_refuses():
    rows = ng.lib().ngram_adamw_rows
    t = ctypes.byref(tensor())
    assert rows(None, 8, 8, A, 4, A, step(), None) == EINVAL
    assert rows(t, 0, 8, A, 4, A, step(), None) == ERANGE and rows(t, 1 << 31, 8, A, 4, A, step(), None) == ERANGE
    assert rows(t, 8, 12, A, 4, A, step(), None) == EINVAL and rows(t, 8, 65544, A, 4, A, step(), None) == ERANGE
    assert rows(t, 8, 8, A, -1, A, step(), None) == EINVAL and rows(t, 8, 8, None, 4, A, step(), None) == EINVAL
    assert rows(t, 8, 8, A + 2, 4, A, step(), None) == EALIGN and rows(t, 8, 8, A, 4, A + 4, step(), None) == EALIGN
    assert rows(t, 8, 8, A, 1 << 31, A, step(), None) == ERANGE
    assert rows(t, 8, 8, None, 0, None, step(), None) == OK


def test_struct_sizes_equal_the_header():
    """The ctypes mirrors have the header's fields in its order."""
    text = open(os.path.join(os.path.dirname(ng.HERE), "include", "ngram.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, cls in (("ngram_fp8", ng._Fp8), ("ngram_adamw_tensor", ng._AdamWTensor), ("ngram_adamw_step", ng._AdamWStep)):
        body = re.search(r"typedef struct \{([^}]*)\}\s*%s;" % name, text).group(1)
        fields = [re.split(r"[\s\*]+", f.strip())[-1] for f in body.split(";") if f.strip()]
        assert fields == [f for f, _ in cls._fields_]
