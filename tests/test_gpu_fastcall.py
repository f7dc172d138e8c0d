"""The binding's short way (_fastcall.so) and its long way give the same bits,
and the short way leaves alone what it should not touch."""
import pytest
import torch

import bit_quantized_moe_softmax_b200 as m

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def fast():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()
    f = m._load_fast()
    assert f is not m._NoFast
    return f


def test_same_results_both_ways(fast, monkeypatch):
    g = torch.Generator(device="cuda").manual_seed(1)
    n, H, V = 5, 264, 1000
    x, res = torch.randn(n, H, generator=g, device="cuda").to(BF16), torch.randn(n, H, generator=g, device="cuda")
    w, W = torch.rand(H, device="cuda"), torch.randn(V, H, generator=g, device="cuda").to(BF16)
    A, B = (torch.randn(2, *s, generator=g, device="cuda").to(BF16) for s in ((8, H), (V, 8)))
    sc, ids = torch.ones(2, device="cuda"), torch.tensor([0, 1, -1, 1, 0], dtype=torch.int32, device="cuda")
    u = torch.rand(n, generator=g, device="cuda")

    def run():
        s, o = torch.empty_like(res), torch.empty(n, H, dtype=BF16, device="cuda")
        q, qs = torch.empty(n, H, dtype=torch.int8, device="cuda"), torch.empty(n, 5, device="cuda")
        wide, y = torch.empty(n, H, device="cuda"), torch.empty(n, V, dtype=BF16, device="cuda")
        t, p, f = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, V, device="cuda")
        m.ds4moe_add_rmsnorm(x, w, 1e-5, residual=res, sum=s, out=o, q=q, scale=qs, group=64)
        m.ds4moe_widen_rows(q, qs, wide, group=64)
        m.ds4moe_project(o, W, y, A=A, B=B, adapter_scale=sc, ids=ids)
        m.ds4moe_sample(y, u, t, temperature=u + 0.5, top_k=ids + 30, top_p=u, min_p=u * 0.01, prob=p, probs=f)
        return s, o, q, qs, wide, y, t, p, f

    short = run()
    monkeypatch.setattr(m, "_fast", m._NoFast)
    for a, b in zip(short, run()):
        assert torch.equal(a, b)


def test_takes_only_what_is_in_order(fast):
    x, w, o = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda"), torch.full((4, 64), 7.0, device="cuda")
    norm = lambda *a: fast.add_rmsnorm(*a)  # noqa: E731
    assert norm(x, w, 1e-6, None, None, o, None, None, 128) and bool((o == 0).all())
    o.fill_(7)
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, 2, device="cuda")
    for bad in ((x.half(), w, 1e-6, None, None, o, None, None, 128), (x, w[:32], 1e-6, None, None, o, None, None, 128),
                (x.cpu(), w, 1e-6, None, None, o, None, None, 128), (x, w, 0.0, None, None, o, None, None, 128),
                (x, w, 1, None, None, o, None, None, 128), (x, w, 1e-6, None, None, o, q, s, 64), (x, w, 1e-6, None, None, o, q, s, 48),
                (x, w, 1e-6, x, x.bfloat16(), o, None, None, 128), (x, w, 1e-6, None, None, o.t(), None, None, 128),
                (x, w, 1e-6, None, None, x, None, None, 128), (None,) * 9, (), (x, "w", 1e-6, None, None, o, None, None, 128)):
        assert norm(*bad) is False
    torch.cuda.synchronize()
    assert bool((o == 7).all())
    b = x.to(BF16)
    assert fast.project(b, b, torch.zeros(4, 4, dtype=BF16, device="cuda"), None, None, None, None)
    assert fast.project(b, b, torch.zeros(4, 4, dtype=BF16, device="cuda"), None, b, None, None) is False
    assert fast.project(b, b[:, :60], torch.zeros(4, 4, dtype=BF16, device="cuda"), None, None, None, None) is False
    assert fast.sample(x.t(), w, w, None, None, None, None, None, None) is False
    assert fast.widen_rows(q, s, o, 64) is False and fast.widen_rows(q, s, o, 32)
