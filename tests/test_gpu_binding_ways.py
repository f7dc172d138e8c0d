"""Both ways through the binding (the compiled one on the current stream, the other
with an explicit stream) take the same calls and refuse the same ones."""
import pytest
import torch

import bit_quantized_moe_softmax_b200 as m

pytestmark = pytest.mark.gpu

F32, BF16, INT8, I32 = torch.float32, torch.bfloat16, torch.int8, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()


def _z(*shape, dtype=F32):
    return torch.ones(*shape, dtype=dtype, device="cuda")


def _both(fn, make):
    """(status, outputs) each way, on its own tensors."""
    got = []
    for stream in (None, torch.cuda.current_stream()):
        args, kw, outs = make()
        try:
            fn(*args, stream=stream, **kw)
            status = 0
        except m.Ds4MoeError as e:
            status = e.status
        torch.cuda.synchronize()
        got.append((status, outs))
    assert got[0][0] == got[1][0], (got[0][0], got[1][0])
    assert all(torch.equal(a, b) for a, b in zip(got[0][1], got[1][1]))
    return got[0][0]


@pytest.mark.parametrize("group, with_q, status", [(48, False, 0), (0, False, 0), (128, False, 0), (1000, False, 0), (-3, False, 0),
                                                   (2 ** 40, False, 0), (48, True, -1), (-1, True, -1), (256, True, -1),
                                                   (64, True, 0), (0, True, 0)])
def test_norms_group(group, with_q, status):
    def make():
        out, q = _z(4, 192), _z(4, 192, dtype=INT8)
        scale = _z(4, 1 if group <= 0 else -(-192 // group) if group <= 192 else 1)
        kw = dict(out=out, group=group, **(dict(q=q, scale=scale) if with_q else {}))
        return (_z(4, 192), _z(192), 1e-6), kw, (out, q, scale)

    assert _both(m.ds4moe_add_rmsnorm, make) == status


@pytest.mark.parametrize("change, status", [({}, 0), (dict(eps=0.0), -1), (dict(eps=1), 0), (dict(residual="x"), 0), (dict(sum="x"), -1),
                                            (dict(residual="x", sum="bf"), -1), (dict(scale="s"), -1), (dict(q="q"), -1),
                                            (dict(out="t"), -1), (dict(out="in"), -1), (dict(weight="short"), -1), (dict(n=0), 0)])
def test_norms_arguments(change, status):
    def make():
        n = change.get("n", 4)
        x = _z(n, 64) * 3
        some = dict(x=_z(n, 64), bf=_z(n, 64, dtype=BF16), s=_z(n, 1), q=_z(n, 64, dtype=INT8), t=_z(64, n).t(), short=_z(32))
        some["in"] = x
        kw = {k: some.get(v, v) if isinstance(v, str) else v for k, v in change.items() if k not in ("eps", "weight", "n")}
        kw.setdefault("out", _z(n, 64))
        w = some["short"] if "weight" in change else _z(64)
        return (x, w, change.get("eps", 1e-6)), kw, (kw["out"],)

    assert _both(m.ds4moe_add_rmsnorm, make) == status


@pytest.mark.parametrize("group, q, out, status", [(128, INT8, F32, 0), (0, INT8, BF16, -1), (48, INT8, F32, -1), (128, F32, F32, -1),
                                                   (128, INT8, INT8, -1)])
def test_widenings_arguments(group, q, out, status):
    def make():
        o = _z(3, 256, dtype=out)
        return (_z(3, 256, dtype=q), _z(3, 2), o), dict(group=group), (o,)

    assert _both(m.ds4moe_widen_rows, make) == status


@pytest.mark.parametrize("adapters, change, status", [(0, {}, 0), (3, {}, 0), (3, dict(ids=None), -1), (3, dict(B=None), -1),
                                                      (3, dict(A=None), -1), (3, dict(rank=12), -3), (0, dict(fin=60), -3)])
def test_projections_arguments(adapters, change, status):
    def make():
        fin, rank = change.get("fin", 64), change.get("rank", 8)
        out = _z(5, 40, dtype=BF16)
        kw = dict(A=_z(3, rank, fin, dtype=BF16), B=_z(3, 40, rank, dtype=BF16), adapter_scale=_z(3), ids=_z(5, dtype=I32)) \
            if adapters else {}
        kw.update({k: v for k, v in change.items() if k in kw})
        return (_z(5, fin, dtype=BF16), _z(40, fin, dtype=BF16), out), kw, (out,)

    assert _both(m.ds4moe_project, make) == status


@pytest.mark.parametrize("change, status", [({}, 0), (dict(u=2), -1), (dict(top_k="f"), -1), (dict(V=(1 << 18) + 1), -3), (dict(n=0), 0)])
def test_samplings_arguments(change, status):
    def make():
        n, V = change.get("n", 2), change.get("V", 50)
        token = _z(n, dtype=I32)
        kw = dict(top_k=_z(n)) if "top_k" in change else {}
        return (_z(n, V), _z(n + 1 if "u" in change else n) * 0.5, token), kw, (token,)

    assert _both(m.ds4moe_sample, make) == status
