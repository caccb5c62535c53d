"""The vocabulary's calls of the C ABI and the binding without a GPU: sizes, and
bad arguments turned away on the host before anything is launched."""
import ctypes
import os
import re

import pytest

import hashed_gram_embedding_ngram_amd as ng

torch = pytest.importorskip("torch")

OK, EINVAL, EALIGN, ERANGE = 0, -1, -2, -3
A = 0x10000             # a fake, aligned device address (never dereferenced)
NAN, INF = float("nan"), float("inf")


def int4(codes=A, scales=A, zeros=A, rows=16, cols=256, group=64, dtype=1):
    return ctypes.byref(ng._Int4(codes, scales, zeros, rows, cols, group, dtype))


def test_sizes():
    L = ng.lib()
    assert L.ngram_int4_code_bytes(3, 40) == 3 * 32 and L.ngram_int4_code_bytes(0, 8) == 0
    assert L.ngram_int4_scales(3, 136, 32) == 3 * 8 and L.ngram_int4_scales(3, 128, 128) == 3 * 4
    for rows, cols in ((-1, 8), (8, -8), (8, 12), ((1 << 24) + 1, 8), (8, (1 << 20) + 8)):
        assert L.ngram_int4_code_bytes(rows, cols) == -1 and L.ngram_int4_scales(rows, cols, 32) == -1
    assert L.ngram_int4_scales(8, 8, 48) == -1
    assert L.ngram_beam_step_workspace_bytes(1, 4, 1000, 0) > 0
    for bad in ((-1, 4, 1000, 0), (1, 0, 1000, 0), (1, 33, 1000, 0), (1, 4, 0, 0), (1, 4, ng.PAD_ID, 0), (1, 4, 1000, 2)):
        assert L.ngram_beam_step_workspace_bytes(*bad) == -1
    assert L.ngram_distill_workspace_bytes(0, 5, 1, 0) >= 0 and L.ngram_distill_workspace_bytes(3, 5, 1, 1) > 0
    for bad in ((-1, 5, 1, 0), (1, 0, 1, 0), (1, (1 << 30) + 1, 1, 0), ((1 << 30) + 1, 5, 1, 0), (1, 5, 1, 2), (1, 5, 0, 0), (1, 5, 1025, 0)):
        assert L.ngram_distill_workspace_bytes(*bad) == -1


BAD_INT4 = [(dict(rows=-1), EINVAL), (dict(cols=12), EINVAL), (dict(cols=-8), EINVAL), (dict(group=16), EINVAL), (dict(dtype=2), EINVAL),
            (dict(rows=(1 << 24) + 1), ERANGE), (dict(cols=(1 << 20) + 8), ERANGE), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL),
            (dict(codes=A + 8), EALIGN), (dict(scales=A + 4), EALIGN), (dict(zeros=A + 2), EALIGN)]


@pytest.mark.parametrize("kw,code", BAD_INT4)
def test_int4_matrices_refused(kw, code):
    L = ng.lib()
    shape = dict(rows=16, cols=256) | {k: v for k, v in kw.items() if k in ("rows", "cols")}
    assert L.ngram_quant_int4(A, 0, shape["rows"], shape["cols"], int4(**kw), None) == code
    assert L.ngram_dequant_int4(int4(**kw), A, 0, None) == code
    assert L.ngram_project_int4(A, 0, 4, int4(**kw), A, 0, None) == code, L.ngram_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(xt=2), EINVAL), (dict(yt=-1), EINVAL), (dict(n=-1), EINVAL), (dict(n=(1 << 30) + 1), ERANGE), (dict(w=None), EINVAL),
    (dict(w=int4(cols=0)), EINVAL), (dict(x=None), EINVAL), (dict(y=None), EINVAL), (dict(x=A + 8), EALIGN), (dict(y=A + 2), EALIGN),
    (dict(n=0, x=None, y=None), OK), (dict(w=int4(rows=0, codes=None)), OK),
])
def test_project_refuses(kw, code):
    a = dict(x=A, xt=1, n=4, w=int4(), y=A, yt=1) | kw
    assert ng.lib().ngram_project_int4(a["x"], a["xt"], a["n"], a["w"], a["y"], a["yt"], None) == code, ng.lib().ngram_last_error()


def test_quant_refuses():
    L = ng.lib()
    assert L.ngram_quant_int4(A, 2, 16, 256, int4(), None) == EINVAL and L.ngram_quant_int4(A, 0, 16, 128, int4(), None) == EINVAL
    assert L.ngram_quant_int4(None, 0, 16, 256, int4(), None) == EINVAL and L.ngram_quant_int4(A + 8, 0, 16, 256, int4(), None) == EALIGN
    assert L.ngram_quant_int4(A, 0, 16, 256, None, None) == EINVAL and L.ngram_quant_int4(None, 0, 0, 256, int4(rows=0), None) == OK
    assert L.ngram_dequant_int4(int4(), A, 3, None) == EINVAL and L.ngram_dequant_int4(int4(), None, 0, None) == EINVAL
    assert L.ngram_dequant_int4(int4(), A + 8, 0, None) == EALIGN and L.ngram_dequant_int4(int4(cols=0), None, 0, None) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), EINVAL), (dict(dtype=5), EINVAL), (dict(beams=0), ERANGE), (dict(beams=33), ERANGE), (dict(V=0), ERANGE),
    (dict(V=ng.PAD_ID, ld=ng.PAD_ID), ERANGE), (dict(ld=999), EINVAL), (dict(end=-2), EINVAL), (dict(end=1000), EINVAL),
    (dict(end=-1), EINVAL), (dict(history=None), EINVAL), (dict(history_out=None), EINVAL), (dict(tokens=None), EINVAL),
    (dict(logits=None), EINVAL), (dict(scores=None), EINVAL), (dict(scores_out=None), EINVAL), (dict(parents_out=None), EINVAL),
    (dict(logits=A + 1), EALIGN), (dict(logits=A + 2, dtype=0), EALIGN), (dict(scores=A + 2), EALIGN), (dict(tokens_out=A + 1), EALIGN),
    (dict(ws=None), EINVAL), (dict(ws=A + 8), EINVAL), (dict(size=64), EINVAL), (dict(batch=0, logits=None, ws=None), OK),
])
def test_beam_step_refuses(kw, code):
    a = dict(logits=A, dtype=1, batch=2, beams=4, V=1000, ld=1000, scores=A, tokens=A, history=A, finished=A, end=2, scores_out=A,
             tokens_out=A, parents_out=A, history_out=A, finished_out=A, ws=A, size=1 << 20) | kw
    assert ng.lib().ngram_beam_step(*a.values(), None) == code, ng.lib().ngram_last_error()


def state(data=A, row=16, stride=16):
    return ng._BeamState(data, row, stride)


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), EINVAL), (dict(batch=-1), EINVAL), (dict(beams=0), ERANGE), (dict(beams=33), ERANGE), (dict(states=None), EINVAL),
    (dict(states=(ng._BeamState * 2)(state(), state(row=-1))), EINVAL), (dict(states=(ng._BeamState * 2)(state(), state(stride=8))), EINVAL),
    (dict(states=(ng._BeamState * 2)(state(), state(row=1 << 41, stride=1 << 41))), ERANGE),
    (dict(states=(ng._BeamState * 2)(state(), state(data=None))), EINVAL), (dict(parents=None), EINVAL), (dict(parents=A + 2), EALIGN),
    (dict(count=0, states=None, parents=None), OK), (dict(batch=0, parents=None), OK),
])
def test_beam_reorder_refuses(kw, code):
    a = dict(states=(ng._BeamState * 2)(state(), state()), count=2, parents=A, batch=3, beams=4) | kw
    assert ng.lib().ngram_beam_reorder(*a.values(), None) == code, ng.lib().ngram_last_error()


BAD_DISTILL = [
    (dict(n=-1), EINVAL), (dict(k=0), EINVAL), (dict(k=1025), ERANGE), (dict(V=0, ld=0), ERANGE), (dict(V=(1 << 30) + 1, ld=1 << 31), ERANGE),
    (dict(ld=99), EINVAL), (dict(dtype=2), EINVAL), (dict(tdtype=-1), EINVAL), (dict(T=0.0), EINVAL), (dict(T=-1.0), EINVAL),
    (dict(T=NAN), EINVAL), (dict(T=INF), EINVAL), (dict(T=1e-40), EINVAL), (dict(z=None), EINVAL), (dict(t=None), EINVAL), (dict(ids=None), EINVAL),
    (dict(z=A + 1), EALIGN), (dict(z=A + 2, dtype=0), EALIGN), (dict(t=A + 1), EALIGN), (dict(ids=A + 2), EALIGN), (dict(lse=A + 2), EALIGN),
]


def distill_args(**kw):
    a = dict(z=A, t=A, ids=A, lse=A, n=4, V=100, ld=100, k=5, dtype=1, tdtype=1, T=1.0) | kw
    return ctypes.byref(ng._DistillArgs(*a.values()))


@pytest.mark.parametrize("kw,code", BAD_DISTILL)
def test_distill_refuses_arguments(kw, code):
    L = ng.lib()
    assert L.ngram_distill(distill_args(**kw), A, A, A, 1.0, None, 0, A, 1 << 20, None) == code, L.ngram_last_error()
    assert L.ngram_distill_grad(distill_args(**kw), A, A, 1.0, A, kw.get("ld", 100), None) in (code, EINVAL), L.ngram_last_error()


def test_distill_refuses():
    f, g, a = ng.lib().ngram_distill, ng.lib().ngram_distill_grad, distill_args()
    ws = (A, 1 << 20, None)
    assert f(None, A, None, None, 1.0, None, 0, *ws) == EINVAL and f(a, None, None, None, 1.0, None, 0, *ws) == EINVAL
    assert f(a, A + 2, None, None, 1.0, None, 0, *ws) == EALIGN and f(a, A, A + 2, None, 1.0, None, 0, *ws) == EALIGN
    assert f(a, A, None, None, 1.0, A + 256, 99, *ws) == EINVAL and f(a, A, None, None, NAN, A + 256, 100, *ws) == EINVAL
    assert f(a, A, None, None, 1.0, A, 101, *ws) == EINVAL                       # in place, but rows apart by another distance
    assert f(a, A, None, A + 1, 1.0, A + 256, 100, *ws) == EALIGN and f(a, A, None, None, 1.0, A + 1, 100, *ws) == EALIGN
    assert f(a, A, None, None, 1.0, None, 0, None, 0, None) == EINVAL and f(a, A, None, None, 1.0, None, 0, A, 8, None) == EINVAL
    assert f(a, A, None, None, 1.0, None, 0, A + 8, 1 << 20, None) == EINVAL
    assert f(distill_args(n=0, z=None), A, None, None, 1.0, None, 0, None, 0, None) == OK
    assert g(a, None, A, 1.0, A, 100, None) == EINVAL and g(a, A, A, 1.0, None, 100, None) == EINVAL
    assert g(a, A, A, INF, A, 100, None) == EINVAL and g(a, A + 2, A, 1.0, A, 100, None) == EALIGN
    assert g(distill_args(n=0), None, None, 1.0, None, 100, None) == OK


def test_struct_fields_equal_the_header():
    text = open(os.path.join(os.path.dirname(ng.HERE), "include", "ngram.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, cls in (("ngram_int4", ng._Int4), ("ngram_beam_state", ng._BeamState), ("ngram_distill_args", ng._DistillArgs)):
        body = re.search(r"typedef struct \{([^}]*)\}\s*%s;" % name, text).group(1)
        fields = [re.split(r"[\s\*]+", f.strip())[-1] for f in body.split(";") if f.strip()]
        assert fields == [f for f, _ in cls._fields_]
    for name, value in (("NGRAM_MAX_BEAMS", ng.MAX_BEAMS), ("NGRAM_DISTILL_MAX_K", ng.DISTILL_MAX_K),
                        ("NGRAM_INT4_MAX_ROWS", ng.INT4_MAX_ROWS), ("NGRAM_INT4_MAX_COLS", ng.INT4_MAX_COLS)):
        assert int(re.search(r"#define %s (\d+)" % name, text).group(1)) == value


class Dev:
    """A tensor's face on a device."""

    def __init__(self, t, device=0, contiguous=True):
        self.t, self.d, self.ok = t, device, contiguous
        self.dtype, self.shape, self.is_cuda, self.device = t.dtype, t.shape, True, torch.device("cuda", device)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, i):
        return self.t[i]

    def get_device(self):
        return self.d

    def is_contiguous(self):
        return self.ok and self.t.is_contiguous()


@pytest.fixture
def no_launch(monkeypatch):
    class Library:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 4096

            def call(*a):
                raise AssertionError(f"{name} was called")
            return call
    monkeypatch.setattr(ng, "lib", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(ng, "_new", lambda rows, cols, dtype, device, stream: Dev(torch.zeros((rows,) if cols is None else (rows, cols), dtype=dtype)))
    monkeypatch.setattr(ng, "_raw_stream", lambda s: 0)


def f32(*shape):
    return Dev(torch.zeros(shape))


def i32(*shape):
    return Dev(torch.zeros(shape, dtype=torch.int32))


def w4(rows=16, cols=64):
    return ng.Int4(Dev(torch.zeros((rows, 32), dtype=torch.uint8)), Dev(torch.zeros((rows, 4))), rows, cols, 64)


OTHER = Dev(torch.zeros(8), device=1)
STREAM1 = type("S", (), {"device_index": 1, "cuda_stream": 0})()


def test_beam_states_overlap(no_launch):
    t = torch.zeros(8, 6)
    for pair in ([t, t], [t[:, :4], t[:, 3:]], [t, t[1:].view(7, 6)[:, :2]], [t[:, 2:], t[:, :3]], [t, t.view(4, 12)], [t, t.view(8, 2, 3)]):
        rows = min(p.shape[0] for p in pair)
        with pytest.raises(ng.NgramError, match="overlap"):
            ng.BeamStates([Dev(p[:rows]) for p in pair])
    for pair in ([t[:, :4], t[:, 4:]], [t[:4], t[4:]], [t[:0], t[:0]], [t[:, :2], t[:, 4:], t[:, 2:4]], [t[:1], t[1:2]], [t[:, :0], t]):
        assert ng.BeamStates([Dev(p) for p in pair]).count == len(pair)


@pytest.mark.parametrize("call,match", [
    (lambda: ng.ngram_project_int4(f32(4, 72), w4()), "columns"),
    (lambda: ng.ngram_project_int4(torch.zeros(4, 64), w4()), "device tensor"),
    (lambda: ng.ngram_project_int4(f32(4, 64), w4(), out=f32(4, 8)), "elements"),
    (lambda: ng.ngram_project_int4(Dev(torch.zeros(4, 64), device=1), w4()), "current"),
    (lambda: ng.ngram_project_int4(f32(4, 64), w4(), stream=STREAM1), "stream of cuda:1"),
    (lambda: ng.Int4(Dev(torch.zeros(4, dtype=torch.uint8)), f32(64), 16, 64), "codes"),
    (lambda: ng.Int4(Dev(torch.zeros((16, 32), dtype=torch.uint8)), Dev(torch.zeros((16, 4)), device=1), 16, 64, 64), "several devices"),
    (lambda: ng.Int4.empty(4, 64, scale_dtype=torch.float16), "fp32 or bf16"),
    (lambda: ng.ngram_quant_int4(f32(4, 64), scale_dtype=torch.float16), "fp32 or bf16"),
    (lambda: ng.BeamStates([f32(8, 3), Dev(torch.zeros(8, 3), device=1)]), "several devices"),
    (lambda: ng.Int4.empty(4, 12), "no 4-bit matrix"), (lambda: ng.Int4.empty(4, 64, 48), "no 4-bit matrix"),
    (lambda: ng.Int4.empty(4, 64, device="cpu"), "lies on a GPU"),
    (lambda: ng.ngram_quant_int4(f32(4, 5, 6)), "two dimensions"),
    (lambda: ng.ngram_beam_step(f32(6, 50), f32(6), 4), "whole sequences"),
    (lambda: ng.ngram_beam_step(f32(4, 50), f32(3), 4), "scores"),
    (lambda: ng.ngram_beam_step(Dev(torch.zeros(50, 4).t()), f32(4), 4), "contiguous"),
    (lambda: ng.ngram_beam_step(Dev(torch.zeros(1, 50).expand(4, 50)), f32(4), 4), "overlap"),
    (lambda: ng.ngram_beam_step(f32(4, 50), f32(4), 4, workspace=torch.zeros(9)), "current"),
    (lambda: ng.ngram_beam_step(f32(4, 50), f32(4), 4, finished=i32(4), end_token=2), "finished"),
    (lambda: ng.ngram_beam_reorder(ng.BeamStates([f32(8, 3)]), i32(4), 4), "4 parents for 8 rows"),
    (lambda: ng.BeamStates([f32(8, 3), f32(4, 3)]), "same rows"),
    (lambda: ng.BeamStates([torch.zeros(8, 3)]), "device tensor"),
    (lambda: ng.BeamStates([Dev(torch.zeros(8, 3, 2).transpose(1, 2))]), "contiguous"),
    (lambda: ng.BeamStates([Dev(torch.zeros(1, 4).expand(8, 4))]), "overlap"),
    (lambda: ng.ngram_distill(f32(4, 50), f32(4, 3), i32(4, 2)), "equal shapes"),
    (lambda: ng.ngram_distill(f32(4, 50), f32(3, 3), i32(3, 3)), "a row for each"),
    (lambda: ng.ngram_distill(f32(4, 50), f32(4, 3), i32(4, 3), dlogits_out=f32(4, 49)), "dlogits_out"),
    (lambda: ng.ngram_distill(f32(4, 50), f32(4, 3), i32(4, 3), teacher_lse=f32(3)), "teacher_lse"),
    (lambda: ng.ngram_distill(f32(4, 50), f32(4, 3), i32(4, 3), weight=OTHER), "current"),
    (lambda: ng.ngram_distill_grad(f32(4, 50), f32(4, 3), i32(4, 3), f32(4)), "stats"),
], ids=range(31))
def test_binding_refuses(call, match, no_launch):
    with pytest.raises(ng.NgramError, match=match):
        call()
