"""Refusals of the operators around the layer, without a GPU: every check of
the C entry points comes before any CUDA call, so plain numbers stand in for
device pointers; the Python binding refuses tensors by type, shape, device and
layout before it calls them."""
import math

import pytest
import torch

import bit_quantized_moe_softmax_b200 as m

A, B, C, D, E, F, G = (0x10000000 * (i + 1) for i in range(7))   # 256-byte aligned, far apart
ARG, ALIGN, SHAPE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_moe_softmax_b200 import build

    build.build()
    return m.lib()


def _norm(lib, **kw):
    a = dict(x=A, xt=0, res=B, rt=0, w=C, eps=1e-6, n=4, H=256, sum=D, out=E, ot=1, q=F, fmt=0, group=128, scale=G)
    a.update(kw)
    return lib.ds4moe_add_rmsnorm(a["x"], a["xt"], a["res"], a["rt"], a["w"], a["eps"], a["n"], a["H"], a["sum"], a["out"],
                                  a["ot"], a["q"], a["fmt"], a["group"], a["scale"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), ARG), (dict(H=0), ARG), (dict(H=16385), SHAPE), (dict(xt=2), ARG), (dict(rt=7), ARG), (dict(ot=-1), ARG),
    (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.inf), ARG), (dict(eps=math.nan), ARG), (dict(fmt=2), ARG),
    (dict(group=16), ARG), (dict(group=256), ARG), (dict(group=-1), ARG), (dict(x=None), ARG), (dict(w=None), ARG),
    (dict(sum=None, out=None, q=None, scale=None), ARG), (dict(res=None), ARG), (dict(q=None), ARG), (dict(scale=None), ARG),
    (dict(x=A + 8), ALIGN), (dict(res=B + 4), ALIGN), (dict(w=C + 4), ALIGN), (dict(sum=D + 8), ALIGN), (dict(out=E + 2), ALIGN),
    (dict(q=F + 1), ALIGN), (dict(scale=G + 2), ALIGN), (dict(out=A), ARG), (dict(sum=A), ARG), (dict(out=B + 16), ARG),
    (dict(q=E + 16), ARG), (dict(scale=C), ARG), (dict(sum=B + 16), ARG), (dict(x=B, sum=B), ARG),
])
def test_add_rmsnorm(lib, kw, status):
    assert _norm(lib, **kw) == status
    assert m.ds4moe_last_error().startswith("add_rmsnorm")


def test_no_rows_is_a_no_op(lib):
    assert _norm(lib, n=0) == 0
    assert lib.ds4moe_widen_rows(None, 0, None, 128, 0, 256, None, 0, None) == 0
    assert lib.ds4moe_project(None, 0, None, 64, 64, None, None, None, 0, 0, None, None, None, 0, None) == 0
    assert lib.ds4moe_sample(None, 0, 10, 0, 10, None, None, None, None, None, None, None, None, None) == 0


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), ARG), (dict(H=0), ARG), (dict(fmt=2), ARG), (dict(group=33), ARG), (dict(ot=2), ARG), (dict(q=None), ARG),
    (dict(scale=None), ARG), (dict(out=None), ARG), (dict(q=A + 8), ALIGN), (dict(out=C + 8), ALIGN), (dict(scale=B + 2), ALIGN),
    (dict(out=A + 512), ARG), (dict(out=B), ARG), (dict(n=1 << 30, H=1 << 20), SHAPE),
])
def test_widen_rows(lib, kw, status):
    a = dict(q=A, fmt=0, scale=B, group=128, n=4, H=256, out=C, ot=0)
    a.update(kw)
    assert lib.ds4moe_widen_rows(a["q"], a["fmt"], a["scale"], a["group"], a["n"], a["H"], a["out"], a["ot"], None) == status
    assert m.ds4moe_last_error().startswith("widen_rows")


def _project(lib, **kw):
    a = dict(x=A, n=4, W=B, fin=64, fout=100, A=C, B=D, s=E, na=3, r=8, ids=E + 4096, out=F, work=G, wb=1 << 20)
    a.update(kw)
    return lib.ds4moe_project(a["x"], a["n"], a["W"], a["fin"], a["fout"], a["A"], a["B"], a["s"], a["na"], a["r"], a["ids"],
                              a["out"], a["work"], a["wb"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), ARG), (dict(n=(1 << 20) + 1), ARG), (dict(fin=0), ARG), (dict(fout=0), ARG), (dict(na=-1), ARG),
    (dict(fin=60), SHAPE), (dict(fin=65544), SHAPE), (dict(fout=(1 << 20) + 1), SHAPE), (dict(na=65537), SHAPE),
    (dict(r=4), SHAPE), (dict(r=20), SHAPE), (dict(r=136), SHAPE), (dict(r=0), SHAPE),
    (dict(x=None), ARG), (dict(W=None), ARG), (dict(out=None), ARG), (dict(A=None), ARG), (dict(B=None), ARG),
    (dict(s=None), ARG), (dict(ids=None), ARG), (dict(work=None), ARG), (dict(wb=0), ARG), (dict(x=A + 8), ALIGN),
    (dict(W=B + 8), ALIGN), (dict(out=F + 2), ALIGN), (dict(A=C + 8), ALIGN), (dict(B=D + 8), ALIGN), (dict(work=G + 16), ALIGN),
    (dict(s=E + 2), ALIGN), (dict(ids=E + 4098), ALIGN), (dict(out=A), ARG), (dict(out=B + 64), ARG), (dict(work=F), ARG),
    (dict(work=D), ARG),
])
def test_project(lib, kw, status):
    assert _project(lib, **kw) == status
    assert m.ds4moe_last_error().startswith("project")


def test_project_work_bytes(lib):
    need = m.ds4moe_project_work_bytes(4, 64, 100, 3, 8)
    assert need > 0 and _project(lib, wb=need - 1) == ARG
    assert m.ds4moe_project_work_bytes(4, 64, 100, 0, 0) == 0
    for bad in ((0, 64, 100, 3, 8), (4, 60, 100, 3, 8), (4, 64, 100, 3, 12), (-1, 64, 100, 3, 8)):
        assert m.ds4moe_project_work_bytes(*bad) == 0


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), ARG), (dict(V=0), ARG), (dict(dt=2), ARG), (dict(V=(1 << 18) + 1, ld=1 << 19), SHAPE), (dict(ld=99), ARG),
    (dict(ld=(1 << 32) + 1), ARG), (dict(n=(1 << 24) + 1), ARG), (dict(l=None), ARG), (dict(u=None), ARG), (dict(tok=None), ARG),
    (dict(l=A + 2), ALIGN), (dict(l=A + 1, dt=1), ALIGN), (dict(u=B + 2), ALIGN), (dict(T=C + 1), ALIGN), (dict(tok=E + 2), ALIGN),
    (dict(probs=G + 2), ALIGN), (dict(tok=A), ARG), (dict(prob=B), ARG), (dict(probs=A + 400), ARG), (dict(prob=E), ARG),
])
def test_sample(lib, kw, status):
    a = dict(l=A, dt=0, ld=100, n=4, V=100, T=C, k=C + 4096, p=C + 8192, mp=D, u=B, tok=E, prob=F, probs=G)
    a.update(kw)
    assert lib.ds4moe_sample(a["l"], a["dt"], a["ld"], a["n"], a["V"], a["T"], a["k"], a["p"], a["mp"], a["u"], a["tok"],
                             a["prob"], a["probs"], None) == status
    assert m.ds4moe_last_error().startswith("sample")


def test_project_error_needs_a_place(lib):
    assert lib.ds4moe_get_project_error(None, None) == ARG


# ------------------------------------------------------------------ the binding
def _z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def _refused(msg, fn, *args, **kw):
    with pytest.raises(m.Ds4MoeError, match=msg) as e:
        fn(*args, **kw)
    assert e.value.status == ARG


def test_binding_refuses_types_shapes_and_devices(lib):
    x, w = _z(4, 64), _z(64)
    norm = m.ds4moe_add_rmsnorm
    _refused("CUDA", norm, x, w, 1e-6, out=x.clone())
    _refused("dimensions", norm, _z(4, 8, 8), w, 1e-6, out=x.clone())
    _refused("x: unsupported type", norm, x.half(), w, 1e-6, out=x.clone())
    _refused("weight: unsupported type", norm, x, w.bfloat16(), 1e-6, out=x.clone())
    _refused("weight: shape", norm, x, _z(63), 1e-6, out=x.clone())
    _refused("group", norm, x, w, 1e-6, q=_z(4, 64, dtype=torch.int8), scale=_z(4, 1), group=48)
    _refused("shape", norm, x, w, 1e-6, q=_z(4, 64, dtype=torch.int8), scale=_z(4, 1), group=32)
    _refused("sum: unsupported type", norm, x, w, 1e-6, residual=x, sum=x.bfloat16())
    _refused("q: unsupported type", m.ds4moe_widen_rows, x, _z(4, 1), x.clone())
    _refused("x: expected", m.ds4moe_project, _z(4), _z(8, 64), _z(4, 8))
    bf = torch.bfloat16
    _refused("need A", m.ds4moe_project, _z(4, 64, dtype=bf), _z(8, 64, dtype=bf), _z(4, 8, dtype=bf), ids=_z(4, dtype=torch.int32))
    _refused("adapters need", m.ds4moe_project, _z(4, 64, dtype=bf), _z(8, 64, dtype=bf), _z(4, 8, dtype=bf),
             A=_z(2, 8, 64, dtype=bf))
    _refused("x: unsupported type", m.ds4moe_project, x, _z(8, 64, dtype=bf), _z(4, 8, dtype=bf))
    _refused("logits: unsupported type", m.ds4moe_sample, x.double(), _z(4), _z(4, dtype=torch.int32))
    _refused("next to each other", m.ds4moe_sample, _z(64, 4).t(), _z(4), _z(4, dtype=torch.int32))
    _refused("u: ", m.ds4moe_sample, x, _z(3), _z(4, dtype=torch.int32))


def test_project_selftest_refuses_as_the_projection_does(lib):
    assert lib.ds4moe_selftest_project_wait(A, 4, B, 64, 100, None, None, None, 0, 0, None, F, None, 0, -1, None) == ARG
    assert lib.ds4moe_selftest_project_wait(A, 4, B, 60, 100, None, None, None, 0, 0, None, F, None, 0, 0, None) == SHAPE
    assert lib.ds4moe_selftest_project_wait(A, 4, B, 64, 100, None, None, None, 0, 0, None, A, None, 0, 0, None) == ARG
