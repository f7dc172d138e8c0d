"""ds4moe_sample against its definition in 64 bits (numpy, row by row).

Tokens and kept sets have to be the same: weights are units of 2^-44 on the
device and binary64 here, so a draw differs only where u or top-p's share falls
within some 2^-40 of a border (fixed seeds).  A probability is at most half a
unit of 2^-44 over the total and one rounding to binary32 off: 2^-24 relative
plus 2^-45 of the largest weight; the bar is 1e-6 relative and 1e-12.
"""
import math

import numpy as np
import pytest
import torch

import bit_quantized_moe_softmax_b200 as m

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()


def reference(logits, u, T=1.0, k=0, p=1.0, mp=0.0):
    """(token, probability, distribution) of one row."""
    l = logits.double().cpu().numpy().copy()
    V = len(l)
    l[np.isnan(l)] = -INF
    probs = np.zeros(V)
    if np.all(l == -INF):
        return -1, 0.0, probs
    order = np.argsort(-l, kind="stable")
    if not T > 0:
        probs[order[0]] = 1.0
        return int(order[0]), 1.0, probs
    top = l[order[0]]
    with np.errstate(all="ignore"):
        w = (l == INF).astype(float) if top == INF else np.where(l == -INF, 0.0, np.exp((l - top) / np.float64(T)))
    if T == INF and top != INF:
        w = (l > -INF).astype(float)
    n = int((l > -INF).sum())
    if 1 <= k < V:
        n = min(n, k)
    f = w[order[:n]]
    if p < 1:
        n = min(n, int(np.searchsorted(np.cumsum(f), max(p, 0.0) * f.sum())) + 1)
    if mp > 0:
        n = min(n, int((f >= min(mp, 1.0)).sum()))
    kept = np.sort(order[:max(n, 1)])
    c = np.cumsum(w[kept])
    u = 0.0 if not u > 0 else u
    j = min(int(np.searchsorted(c, u * c[-1], side="right")), int(np.flatnonzero(w[kept] > 0)[-1]))
    probs[kept] = w[kept] / c[-1]
    return int(kept[j]), float(probs[kept[j]]), probs


def _param(v, n, dtype=F32):
    return None if v is None else torch.as_tensor(v, dtype=dtype).expand(n).contiguous().cuda()


def _check(logits, u, T=None, k=None, p=None, mp=None, probs=True):
    n, V = logits.shape
    dev = logits if logits.is_cuda else logits.cuda()
    T_, k_, p_, mp_, u_ = _param(T, n), _param(k, n, torch.int32), _param(p, n), _param(mp, n), _param(u, n)
    token = torch.full((n + 1,), -5, dtype=torch.int32, device="cuda")
    prob = torch.full((n + 1,), -5.0, device="cuda")
    full = torch.full((n + 1, V), -5.0, device="cuda") if probs else None
    m.ds4moe_sample(dev, u_, token[:n], temperature=T_, top_k=k_, top_p=p_, min_p=mp_, prob=prob[:n],
                    probs=full[:n] if probs else None)
    torch.cuda.synchronize()
    assert int(token[n]) == -5 and float(prob[n]) == -5 and (not probs or bool((full[n] == -5).all())), "behind the last row"
    for i in range(n):
        t, pr, dist = reference(dev[i], float(u_[i]), 1.0 if T is None else float(T_[i]), 0 if k is None else int(k_[i]),
                                1.0 if p is None else float(p_[i]), 0.0 if mp is None else float(mp_[i]))
        assert int(token[i]) == t, (i, int(token[i]), t)
        assert abs(float(prob[i]) - pr) <= 1e-6 * pr + 1e-12, i
        if probs:
            got = full[i].double().cpu().numpy()
            assert np.all(np.abs(got - dist) <= 1e-6 * dist + 1e-12), i
            tiny = dist.max() * 2.0 ** -43   # weights under a unit of 2^-44 may round to nothing
            assert np.array_equal(got > tiny, dist > tiny), i
    return token[:n], prob[:n]


def _logits(n, V, dtype=F32, spread=2.5, seed=0):
    g = torch.Generator().manual_seed(seed + 13 * V + n)
    return (torch.randn(n, V, generator=g) * spread).to(dtype), torch.rand(n, generator=g)


FILTERS = [dict(), dict(k=1), dict(k=7), dict(k=300), dict(p=0.3), dict(p=0.95), dict(mp=0.05), dict(k=40, p=0.8, mp=0.02),
           dict(k=2, p=0.999), dict(T=0.6, p=0.9), dict(T=1.7, k=100, p=0.5)]


@pytest.mark.parametrize("V", [1, 2, 31, 33, 128, 1000, 2048, 8192, 8193, 20001, 40000, 131072])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_vocabularies(V, dtype):
    for i, f in enumerate(FILTERS):
        l, u = _logits(3, V, dtype, seed=i)
        _check(l, u, **f)


@pytest.mark.parametrize("V", [100001, 262144])
def test_largest_vocabularies(V):
    l, u = _logits(2, V, F32)
    for f in (dict(), dict(k=50, p=0.9, mp=0.01), dict(p=0.99)):
        _check(l, u, **f)


def test_batch_of_mixed_requests():
    n, V = 90, 5003
    l, u = _logits(n, V, BF16)
    g = torch.Generator().manual_seed(3)
    T = torch.rand(n, generator=g) * 1.5
    T[::7] = 0
    k = torch.randint(-2, 200, (n,), generator=g)
    p = torch.rand(n, generator=g) * 1.2
    mp = torch.rand(n, generator=g) * 0.1 - 0.02
    _check(l, u, T=T, k=k, p=p, mp=mp)


@pytest.mark.parametrize("T", [0.0, -1.0, NAN, 1e-45, 1e-30, 1e-9, 1e-3, 30.0, 1e6, 3e38, INF])
def test_temperatures(T):
    for V in (300, 20000):
        l, u = _logits(3, V)
        _check(l, u, T=T)
        _check(l, u, T=T, k=20, p=0.7)
        _check(l, u, T=T, p=0.4, mp=0.3)


@pytest.mark.parametrize("f", [dict(k=0), dict(k=-3), dict(k=10 ** 6), dict(p=0.0), dict(p=-1.0), dict(p=1.0), dict(p=7.0),
                               dict(p=NAN), dict(mp=0.0), dict(mp=-1.0), dict(mp=1.0), dict(mp=5.0), dict(mp=NAN), dict(p=1e-30),
                               dict(p=0.99999994), dict(mp=1e-30)])
def test_filters_at_their_ends(f):
    l, u = _logits(4, 777)
    _check(l, u, **f)


@pytest.mark.parametrize("u", [0.0, -1.0, NAN, 1e-30, 0.5, 0.99999994, 1.0, 2.0])
def test_uniform_numbers_at_their_ends(u):
    l, _ = _logits(3, 900)
    _check(l, u)
    _check(l, u, k=5)


@pytest.mark.parametrize("V", [50, 9000, 70000])
def test_ties(V):
    """Equal logits: the lowest indices are kept, across warps and CTAs; an even row of one value, rows of two."""
    g = torch.Generator().manual_seed(V)
    l = torch.zeros(6, V)
    l[1] = torch.randint(0, 2, (V,), generator=g).float()
    l[2] = torch.randint(0, 5, (V,), generator=g).float() / 4
    l[3, ::2] = -0.0
    l[4] = torch.randint(-1, 1, (V,), generator=g).float() * 40
    l[5] = -3e38
    u = torch.rand(6, generator=g)
    for f in (dict(), dict(k=1), dict(k=V // 3), dict(k=V - 1), dict(p=0.5), dict(k=V // 2 + 3, p=0.7), dict(T=0.5, p=0.99),
              dict(mp=1.0), dict(T=0.0)):
        _check(l, u, **f)


@pytest.mark.parametrize("V", [40, 30000])
def test_masked_and_broken_logits(V):
    l, u = _logits(8, V)
    l[0] = -INF
    l[1, : V - 1] = -INF
    l[2, ::2] = -INF
    l[3, 5] = NAN
    l[4] = NAN
    l[5, [3, V - 2]] = INF
    l[6] = torch.finfo(F32).min
    l[7, : V // 2] = torch.finfo(F32).min
    for f in (dict(), dict(k=3), dict(p=0.6), dict(k=V - 1, p=0.9, mp=0.01), dict(T=0.0), dict(T=INF), dict(T=1e-3, k=10)):
        _check(l, u, **f)
    _check(l.to(BF16), u, k=4, p=0.9)


@pytest.mark.parametrize("k", [63, 64, 500, 511, 512, 513, 700])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_top_k_about_a_ctas_threads(k, dtype):
    """Where the kept tokens stop fitting one per thread; bf16's ties put many at the threshold."""
    for V in (1000, 30000, 140000):
        l, u = _logits(2, V, dtype, seed=k)
        for f in (dict(k=k), dict(k=k, p=0.97), dict(k=k, T=0.3, mp=0.1), dict(k=k, T=3.0, p=0.5)):
            _check(l, u, **f)


@pytest.mark.parametrize("spread", [0.01, 1.0, 4.0, 12.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nuclei_of_all_sizes(spread, dtype):
    """Flat and peaked rows: top-p keeps from one token to nearly all of them."""
    for V in (700, 25000, 131072):
        l, u = _logits(3, V, dtype, spread=spread, seed=int(10 * spread))
        for p in (0.05, 0.5, 0.9, 0.999):
            _check(l, u, p=p)
            _check(l, u, p=p, k=2000, mp=0.003, probs=False)


@pytest.mark.parametrize("T", [1.0, 1e36, 3e38, INF])
def test_logits_over_the_whole_range(T):
    """Differences of logits beyond binary32's largest value."""
    l, u = _logits(4, 3000)
    l *= 1e37
    l[:, 7] = 3.3e38
    l[:, 11::5] = torch.finfo(F32).min
    for f in (dict(), dict(k=9), dict(p=0.5), dict(k=2000, p=0.9, mp=0.01)):
        _check(l, u, T=T, **f)


@pytest.mark.parametrize("dtype, pad, start", [(F32, 0, 1), (F32, 3, 2), (BF16, 5, 0), (BF16, 8, 1), (BF16, 1, 3)])
def test_strided_and_unaligned_rows(dtype, pad, start):
    V = 5000
    l, u = _logits(4, V + pad + start, dtype)
    view = l.cuda()[:, start:start + V]
    _check(view, u, k=30, p=0.9)


def test_draws_follow_the_distribution():
    """u in even steps: each kept token is drawn for as many steps as its share, to one."""
    V, n = 200, 4096
    l, _ = _logits(1, V)
    u = (torch.arange(n) + 0.5) / n
    token, _ = _check(l.expand(n, V).contiguous(), u, k=12, p=0.95, probs=False)
    _, _, dist = reference(l[0], 0.0, 1.0, 12, float(np.float32(0.95)))
    count = torch.bincount(token.long().cpu(), minlength=V).numpy()
    assert np.all(np.abs(count - dist * n) <= 1.0)
    assert bool((token[1:] >= token[:-1]).all())


def test_streams_graphs_and_two_calls_at_once():
    l, u = _logits(5, 60000)
    token, prob = _check(l, u, k=80, p=0.9)
    dl, du = l.cuda(), u.cuda()
    k, p = _param(80, 5, torch.int32), _param(0.9, 5)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty(5, dtype=torch.int32, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o in zip(streams, outs):
            m.ds4moe_sample(dl, du, o, top_k=k, top_p=p, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, token) for o in outs)
    g = torch.cuda.CUDAGraph()
    outs[0].zero_()
    with torch.cuda.graph(g):
        m.ds4moe_sample(dl, du, outs[0], top_k=k, top_p=p)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], token)
    dl.copy_(torch.roll(dl, 1, dims=1))   # new logits in the captured buffer
    g.replay()
    torch.cuda.synchronize()
    _check(dl, u, k=80, p=0.9, probs=False)


def test_refusals_on_the_device():
    l, u, t = torch.zeros(2, 8, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(logits=l.half()), dict(u=u.double()), dict(token=t.long()), dict(prob=u), dict(top_k=u), dict(top_p=t),
                dict(probs=torch.zeros(2, 9, device="cuda")), dict(u=u.cpu()), dict(logits=l[:1].expand(2, 8))):
        with pytest.raises(m.Ds4MoeError):
            m.ds4moe_sample(**{**dict(logits=l, u=u, token=t), **bad})
