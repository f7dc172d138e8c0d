"""The binding of the operators around the layer, without a GPU: what becomes of the
short way's answer."""
import os
import sys
import types
import warnings

import pytest
import torch

import bit_quantized_moe_softmax_b200 as m


def _calls():
    x = torch.zeros(2, 8)
    bf, i = x.bfloat16(), torch.zeros(2, dtype=torch.int32)
    return [("add_rmsnorm", lambda: m.ds4moe_add_rmsnorm(x, x[0], 1e-6, out=x.clone())),
            ("widen_rows", lambda: m.ds4moe_widen_rows(x.to(torch.int8), x[:, :1].contiguous(), x.clone())),
            ("project", lambda: m.ds4moe_project(bf, bf.clone(), bf.clone())),
            ("sample", lambda: m.ds4moe_sample(x, x[:, 0].contiguous(), i))]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bit_quantized_moe_softmax_b200 import build

    build.build()


@pytest.mark.parametrize("which", range(4))
def test_a_failure_behind_the_checks_is_raised_and_the_call_not_repeated(monkeypatch, which):
    """The norm adds into its residual in place: a second launch would add twice."""
    name, call = _calls()[which]
    seen = []

    def fails(*args):
        seen.append(name)
        return -5   # DS4MOE_ERR_CUDA

    monkeypatch.setattr(m, "_fast", types.SimpleNamespace(**{name: fails}))
    monkeypatch.setattr(m, "_call", lambda *args: seen.append("again"))
    monkeypatch.setattr(m, "_tensors", lambda *args: None)
    with pytest.raises(m.Ds4MoeError) as e:
        call()
    assert e.value.status == -5 and seen == [name]


@pytest.mark.parametrize("which", range(4))
def test_done_and_not_in_order(monkeypatch, which):
    name, call = _calls()[which]
    for answer, long_way in ((True, []), (False, ["long"])):
        seen = []
        monkeypatch.setattr(m, "_fast", types.SimpleNamespace(**{name: lambda *args: answer}))
        monkeypatch.setattr(m, "_call", lambda *args: seen.append("long"))
        monkeypatch.setattr(m, "_tensors", lambda *args: None)
        call()
        assert seen == long_way


def test_group_means_nothing_without_codes():
    """Refused for being no CUDA tensors, and not for a group that nothing uses."""
    x = torch.zeros(2, 64)
    with pytest.raises(m.Ds4MoeError, match="CUDA"):
        m.ds4moe_add_rmsnorm(x, x[0], 1e-6, out=x.clone(), group=48)
    with pytest.raises(m.Ds4MoeError, match="group"):
        m.ds4moe_add_rmsnorm(x, x[0], 1e-6, q=x.to(torch.int8), scale=x[:, :2].contiguous(), group=48)


def test_sizes_beyond_32_bits_are_refused():
    """2^32 + 4 rows are not 4 rows (tensors without memory stand in)."""
    def z(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="meta")

    n, bf, i32 = 2 ** 32 + 4, torch.bfloat16, torch.int32
    for call in (lambda: m.ds4moe_add_rmsnorm(z(n, 64), z(64), 1e-6, out=z(n, 64)),
                 lambda: m.ds4moe_add_rmsnorm(z(4, n), z(n), 1e-6, out=z(4, n)),
                 lambda: m.ds4moe_widen_rows(z(n, 64, dtype=torch.int8), z(n, 1), z(n, 64)),
                 lambda: m.ds4moe_project(z(n, 64, dtype=bf), z(8, 64, dtype=bf), z(n, 8, dtype=bf)),
                 lambda: m.ds4moe_project(z(4, 64, dtype=bf), z(n, 64, dtype=bf), z(4, n, dtype=bf)),
                 lambda: m.ds4moe_project(z(4, 64, dtype=bf), z(8, 64, dtype=bf), z(4, 8, dtype=bf), A=z(n, 8, 64, dtype=bf),
                                          B=z(n, 8, 8, dtype=bf), adapter_scale=z(n), ids=z(4, dtype=i32)),
                 lambda: m.ds4moe_sample(z(n, 64), z(n), z(n, dtype=i32)), lambda: m.ds4moe_sample(z(4, n), z(4), z(4, dtype=i32))):
        with pytest.raises(m.Ds4MoeError, match="32 bits") as e:
            call()
        assert e.value.status == -1
    assert m.ds4moe_project_work_bytes(4, 64, 100, 3, 8) > 0
    for bad in ((n, 64, 100, 3, 8), (4, 2 ** 32 + 64, 100, 3, 8), (4, 64, 100, 2 ** 32 + 3, 8), (4, 64, 100, 3, 2 ** 32 + 8)):
        assert m.ds4moe_project_work_bytes(*bad) == 0


# ------------------------------------------------------------------ the compiled way's file
def test_compiled_way_is_of_this_python_and_torch(monkeypatch):
    from bit_quantized_moe_softmax_b200 import build

    path = build.fast_path()
    assert torch.__version__ in path and sys.implementation.cache_tag in path and path.endswith(".so")
    assert os.path.exists(path)
    monkeypatch.setattr(m, "_fast", None)
    assert m._load_fast() is not m._NoFast and m._fast.add_rmsnorm() is False
    monkeypatch.setattr(torch, "__version__", "0.0")   # another torch: its file is not there, this one's is not loaded
    monkeypatch.setattr(m, "_fast", None)
    assert build.fast_path() != path and m._load_fast() is m._NoFast


@pytest.mark.parametrize("content", [b"", b"no library", b"\x7fELF" + bytes(200)])
def test_a_file_that_does_not_load_leaves_the_long_way(monkeypatch, tmp_path, content):
    from bit_quantized_moe_softmax_b200 import build

    path = tmp_path / "_fastcall.so"
    path.write_bytes(content)
    monkeypatch.setattr(build, "fast_path", lambda: str(path))
    monkeypatch.setattr(m, "_fast", None)
    x = torch.zeros(2, 8)
    with pytest.warns(UserWarning, match="check in Python"), pytest.raises(m.Ds4MoeError, match="CUDA"):
        m.ds4moe_add_rmsnorm(x, x[0], 1e-6, out=x.clone())
    with warnings.catch_warnings():   # said once
        warnings.simplefilter("error")
        with pytest.raises(m.Ds4MoeError, match="CUDA"):
            m.ds4moe_widen_rows(x.to(torch.int8), x[:, :1].contiguous(), x.clone())
