"""ds4moe_add_rmsnorm and ds4moe_widen_rows against their definitions.

The definition rounds in binary32 at stated points and takes the mean square
in binary64, so a CPU restatement gives the same bits: sums, norms, scales and
8-bit codes are compared for equality (two binary64 sums of one row, each off
by at most 16384 half steps of 2^-53, round to different binary32 reciprocals
once in some 10^5 rows at the very most; the few thousand rows here have fixed
seeds).
"""
import numpy as np
import pytest
import torch

import bit_quantized_moe_softmax_b200 as m
from bit_quantized_moe_softmax_b200 import ep, synth
from tests._util import pack_with_oracle

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()


def _spread(scale, group, H):
    return scale.repeat_interleave(group or H, 1)[:, :H]


def _quantize(y, dtype, group):
    H = y.shape[1]
    qmax = torch.tensor(448.0 if dtype == E4M3 else 127.0)
    scale = torch.stack([p.abs().amax(1) for p in y.split(group or H, dim=1)], 1) / qmax
    s = _spread(scale, group, H)
    t = torch.where(s > 0, y / s, torch.zeros(()))
    return (t.round() if dtype == INT8 else t).to(dtype), scale


def _reference(x, res, w, eps=EPS):
    """(sum, y) by the definition, on the CPU."""
    s = x.float()
    if res is not None:
        s = (s + res.float()).to(res.dtype)
    v = s.float()
    ms = v.double().square().sum(1, keepdim=True) / v.shape[1] + float(np.float32(eps))
    return s, v * (1.0 / ms.sqrt()).float() * w


def _data(n, H, xt, rt, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * n + H)
    x = (torch.randn(n, H, generator=g) * 2).to(xt)
    res = None if rt is None else (torch.randn(n, H, generator=g) * torch.rand(1, H, generator=g) * 3).to(rt)
    return x, res, torch.rand(H, generator=g) + 0.5


def _run(x, res, w, out=None, q=None, group=128, sum_to=None, stream=None, eps=EPS):
    """Device outputs (sum, out, q, scale) as CPU tensors; every buffer has a guard row that has to stay."""
    n, H = x.shape
    dev = {}

    def buf(name, shape, dtype):
        t = torch.full((shape[0] + 1,) + shape[1:], 77, dtype=torch.float32, device="cuda").to(dtype)
        dev[name] = t
        return t[:shape[0]]

    groups = -(-H // group) if group else 1
    kw = dict(residual=None if res is None else res.cuda(), group=group, stream=stream)
    if res is not None:
        kw["sum"] = kw["residual"] if sum_to == "residual" else buf("sum", (n, H), res.dtype)
    if out is not None:
        kw["out"] = buf("out", (n, H), out)
    if q is not None:
        kw["q"], kw["scale"] = buf("q", (n, H), q), buf("scale", (n, groups), F32)
    m.ds4moe_add_rmsnorm(x.cuda(), w.cuda(), eps, **kw)
    torch.cuda.synchronize()
    for t in dev.values():
        assert bool((t[-1].float() == torch.tensor(77.0).to(t.dtype).float().item()).all()), "rows behind the last one"
    return [None if kw.get(k) is None else kw[k].cpu() for k in ("sum", "out", "q", "scale")]


def _same(a, b):
    """Equal bits up to the sign and payload of NaN."""
    a, b = a.float(), b.float()
    assert a.shape == b.shape
    assert bool(((a == b) | (a.isnan() & b.isnan())).all()), (a - b).abs().max()


WIDTHS = [1, 7, 8, 31, 64, 100, 256, 257, 520, 1000, 1024, 2050, 4096, 5000, 8192, 8200, 16384]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("xt, rt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32), (F32, None), (BF16, None)])
def test_norm_widths_and_types(H, xt, rt):
    x, res, w = _data(5, H, xt, rt)
    s, y = _reference(x, res, w)
    for out in (F32, BF16):
        gs, gy, _, _ = _run(x, res, w, out=out)
        _same(gy, y.to(out))
        if rt is not None:
            _same(gs, s)


@pytest.mark.parametrize("H", [1, 31, 40, 64, 129, 250, 256, 1000, 2048, 4096, 4100, 16384])
@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_norm_codes_and_widening(H, dtype, group):
    x, res, w = _data(3, H, F32, BF16, seed=1)
    s, y = _reference(x, res, w)
    q, scale = _quantize(y, dtype, group)
    gs, _, gq, gscale = _run(x, res, w, q=dtype, group=group)
    _same(gs, s)
    _same(gscale, scale)
    _same(gq, q)
    for out in (F32, BF16):
        o = torch.full((4, H), 5.0, device="cuda", dtype=out)
        m.ds4moe_widen_rows(gq.cuda(), gscale.cuda(), o[:3], group=group)
        _same(o[:3].cpu(), (q.float() * _spread(scale, group, H)).to(out))
        assert bool((o[3] == 5).all())
    # the value that a code stands for is at most half a step off (e4m3: 2^-4 of the value, at its smallest scale
    # 2^-10 of a code; int8: half a code), and the division and product round once each
    err = (q.double() * _spread(scale.double(), group, H) - y.double()).abs()
    step = torch.maximum(y.double().abs() * 2.0 ** -4, _spread(scale.double(), group, H) * 2.0 ** -10) if dtype == E4M3 \
        else _spread(scale.double(), group, H) * 0.5
    assert bool((err <= step * (1 + 1e-4) + y.double().abs() * 2.0 ** -22).all())


@pytest.mark.parametrize("n, H", [(1, 4096), (2, 256), (148, 4096), (295, 512), (296, 4096), (700, 300), (2000, 64)])
def test_norm_row_counts(n, H):
    x, res, w = _data(n, H, F32, F32, seed=2)
    s, y = _reference(x, res, w)
    q, scale = _quantize(y, E4M3, 128)
    gs, gy, gq, gscale = _run(x, res, w, out=BF16, q=E4M3)
    _same(gs, s), _same(gy, y.to(BF16)), _same(gq, q), _same(gscale, scale)


def test_sum_in_place_and_stream_and_graph():
    x, res, w = _data(9, 4096, BF16, F32, seed=3)
    s, y = _reference(x, res, w)
    st = torch.cuda.Stream()
    gs, gy, _, _ = _run(x, res, w, out=F32, sum_to="residual", stream=st)
    _same(gs, s), _same(gy, y)
    dx, dr, dw, o = x.cuda(), res.cuda(), w.cuda(), torch.empty(9, 4096, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.ds4moe_add_rmsnorm(dx, dw, EPS, residual=dr, sum=dr, out=o)
    for _ in range(2):   # the captured call updates the stream in place: x + (x + res) at the second replay
        g.replay()
    torch.cuda.synchronize()
    s2, y2 = _reference(x, s, w)
    _same(dr.cpu(), s2), _same(o.cpu(), y2)


def test_extreme_rows():
    """Zero rows, tiny and huge values, infinities and NaN: a row's neighbours do not notice."""
    H = 512
    x = torch.randn(8, H, generator=torch.Generator().manual_seed(5))
    x[1] = 0
    x[2] = 1e-38
    x[3] *= 1e37
    x[4, 100] = float("inf")
    x[5, 7] = float("nan")
    x[6] = -0.0
    w = torch.ones(H)
    s, y = _reference(x, torch.zeros_like(x), w)
    for dtype in (E4M3, INT8):
        gs, gy, gq, gscale = _run(x, torch.zeros_like(x), w, out=F32, q=dtype)
        _same(gs, s), _same(gy, y)
        q, scale = _quantize(y, dtype, 128)
        fine = [0, 1, 2, 3, 6, 7]
        _same(gq[fine], q[fine]), _same(gscale[fine], scale[fine])
        assert bool((gscale[[1, 6]] == 0).all()) and bool((gq[[1, 6]].float() == 0).all())
        wide = torch.empty(8, H, device="cuda")
        m.ds4moe_widen_rows(gq.cuda(), gscale.cuda(), wide)
        wide = wide.cpu()
        assert bool(torch.isfinite(wide[fine]).all())
        bad = ~torch.isfinite(y)
        for r in (4, 5):   # a group with a value that is not finite widens to NaN throughout
            for c in range(0, H, 128):
                assert bool(wide[r, c:c + 128].isnan().all()) == bool(bad[r, c:c + 128].any())


def test_extreme_eps():
    x = torch.zeros(2, 64)
    x[1] = 1e-3
    for eps in (1e-30, 1.0, 3e38):
        _, y = _reference(x, None, torch.ones(64), eps)
        _same(_run(x, None, torch.ones(64), out=F32, eps=eps)[1], y)


def test_widening_beyond_32_bit_indices():
    """n * H above 2^32: the last rows of 8-bit codes land where they belong."""
    n, H = (1 << 20) + 3, 4096
    q = torch.ones(n, H, dtype=INT8, device="cuda")
    q[-1, -5:] = 3
    scale = torch.arange(n, device="cuda", dtype=F32)[:, None] % 251
    out = torch.empty(n, H, dtype=BF16, device="cuda")
    m.ds4moe_widen_rows(q, scale.contiguous(), out, group=0)
    for r in (0, 250, 251, (1 << 20) - 1, n - 2):
        assert bool((out[r] == r % 251).all()), r
    assert bool((out[-1, :-5] == (n - 1) % 251).all()) and bool((out[-1, -5:] == torch.tensor(3.0 * ((n - 1) % 251)).bfloat16()
                                                                .item()).all())


def test_layers_experts_on_8_bit_rows(orc):
    """The norm's 8-bit rows through the expert-parallel step on one process: the experts get exactly the widened
    rows, and the slot-order combine adds their outputs to the base."""
    H, E, k, n = 256, 8, 2, 6
    L = synth.float_layer(synth.Shape(H=H, I=128, E=E, k=k), 3)
    L.update(pack_with_oracle(orc, L))
    shard = ep.GpuExpertShard(L, E, 0, 1, 8)
    x, res, w = _data(n, H, F32, F32, seed=6)
    q = torch.empty(n, H, dtype=E4M3, device="cuda")
    scale = torch.empty(n, 2, device="cuda")
    m.ds4moe_add_rmsnorm(x.cuda(), w.cuda(), EPS, residual=res.cuda(), q=q, scale=scale)
    g = torch.Generator().manual_seed(8)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(n)]).cuda()
    wts, base = torch.rand(n, k, generator=g).cuda(), torch.randn(n, H, generator=g).cuda()
    out = ep.moe_forward_ep_q8(q, scale, ids, wts, E, shard.forward_q8, base, combine_fn=ep.combine_gpu)
    wide = torch.empty(n, H, device="cuda")
    m.ds4moe_widen_rows(q, scale, wide)
    ref = ep.combine_gpu(shard(*ep.dispatch(wide, ids, ep.plan(ids, E))), wts, ep.plan(ids, E), base)
    assert torch.equal(out, ref)
