"""ds4moe_sample on many rows at once, where the CTAs of a row start apart from each
other, against torch on the device; and on logits far apart, against the 64-bit
reference."""
import pytest
import torch

import bit_quantized_moe_softmax_b200 as m
from tests.test_gpu_sample import _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()


@pytest.mark.parametrize("V, n", [(8193, 3000), (8200, 3000), (16385, 2000), (32769, 1000), (65537, 4)])
def test_maximum_in_any_share(V, n):
    """Rows split over 2 to 16 CTAs, each CTA's share as short as the split has it: whichever holds the row's
    largest logit, all the others learn of it."""
    g = torch.Generator(device="cuda").manual_seed(V)
    l = torch.randn(n, V, generator=g, device="cuda")
    at = torch.randint(0, V, (n,), generator=g, device="cuda")
    l[torch.arange(n, device="cuda"), at] = 50.0
    u = torch.rand(n, generator=g, device="cuda")
    zero = torch.zeros(n, device="cuda")
    token, prob = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
    for temperature in (zero, None):   # greedy; and a weight beside which the others' are under 2^-44
        for _ in range(5):
            token.fill_(-7)
            m.ds4moe_sample(l, u, token, temperature=temperature, top_p=None if temperature is zero else zero + 0.5, prob=prob)
            assert torch.equal(token.long(), at) and bool((prob == 1).all())


@pytest.mark.parametrize("T", [1.0, 1e30, 1e36, 1e37, 3e38, float("inf")])
@pytest.mark.parametrize("V", [40, 9000])
def test_largest_logit_beside_the_lowest(V, T):
    """Row maxima from 1e29 to binary32's largest beside tokens at its lowest value, whose difference binary32 cannot
    hold, at temperatures that give them weight all the same."""
    tops = [1e29, 1e31, 1e32, 5e36, 1e37, 1.1e37, 1e38, 3.4e38, -1e32, 5.0]
    l = torch.randn(len(tops), V, generator=torch.Generator().manual_seed(V))
    l[:, 2::3] = torch.finfo(torch.float32).min
    for i, top in enumerate(tops):
        l[i, 1::3] = top * (1 - 0.5 * torch.rand(l[i, 1::3].shape, generator=torch.Generator().manual_seed(i)))
        l[i, 7] = top if top > 0 else 6.0
    u = torch.linspace(0.03, 0.98, len(tops))
    for f in (dict(), dict(k=V // 2), dict(p=0.6), dict(k=V - 3, p=0.9, mp=0.01)):
        _check(l, u, T=T, **f)


def test_order_of_tiny_logits_beside_a_huge_one():
    """Neighbours in binary32 keep their order, however large the row's maximum."""
    V = 600
    l = (torch.arange(V, dtype=torch.int32) + 1).view(torch.float32).repeat(3, 1)   # the smallest subnormals, ascending
    l[:, 0] = torch.tensor([2e37, 3e38, 1.0])
    for k in (3, 40):
        _check(l, torch.tensor([0.999, 0.999, 0.5]), T=float("inf"), k=k)


@pytest.mark.parametrize("T", [1e-45, 3e-42, 1e-38, 2e-37, 1e-33, 1e-29, 2e-29])
@pytest.mark.parametrize("V", [13, 700, 20000])
def test_tiny_temperatures_of_tiny_logits(T, V):
    """Only (l - M) / T counts: logits of the temperature's own size share the weight, down to binary32's last steps;
    beside them tokens that are far below, and a maximum far above."""
    l = torch.randn(4, V, generator=torch.Generator().manual_seed(V), dtype=torch.float64) * 2
    l = (l * float(torch.tensor(T))).float()
    l[1, ::3] = -1e5
    l[2, 1::4] = torch.finfo(torch.float32).min
    l[3, V // 2] = 1e12
    u = torch.tensor([0.1, 0.5, 0.9, 0.7])
    for f in (dict(), dict(k=9), dict(p=0.8), dict(k=V - 2, p=0.9, mp=0.01)):
        _check(l, u, T=T, **f)


@pytest.mark.parametrize("V", [20, 900, 40000])
@pytest.mark.parametrize("f", [dict(), dict(top_k=7), dict(top_k=700), dict(top_p=0.9), dict(top_k=15, top_p=0.9999)])
@pytest.mark.parametrize("T", [1.0, 1e16, 3e38])
def test_min_p_of_one_keeps_the_maximum_alone(V, f, T):
    """Tokens whose weight rounds to 1 in binary64 without being at the maximum are not kept."""
    n = 3
    l = torch.zeros(n, V) if T > 1 else torch.full((n, V), 1e-18)
    l[:, 5::2] = -1e-17 if T == 1 else -0.5
    l[0, 9], l[1, [7, 11]] = (1e-17, 2e-17) if T == 1 else (0.25, 0.5)
    l[2] = torch.finfo(torch.float32).min
    at = [[9], [7, 11], list(range(V))]
    p = {k: torch.full((n,), v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in f.items()}
    token, prob, probs = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, V, device="cuda")
    u = torch.tensor([0.99, 0.25, 0.0], device="cuda")
    m.ds4moe_sample(l.cuda(), u, token, temperature=torch.full((n,), T, device="cuda"), min_p=torch.ones(n, device="cuda"),
                    prob=prob, probs=probs, **p)
    for i in range(n):
        kept = at[i]
        if i == 2:   # all alike: top-k's or top-p's share of them, from the lowest index on
            kept = kept[:f.get("top_k", V)]
            if "top_p" in f:
                kept = kept[:int((probs[i] > 0).sum())]
                assert abs(len(kept) / min(V, f.get("top_k", V)) - f["top_p"]) <= 1.0 / len(kept)
        want = torch.zeros(V)
        want[kept] = 1.0 / len(kept)
        assert int(token[i]) in kept and torch.allclose(probs[i].cpu(), want, rtol=2.0 ** -22, atol=0), i
        assert int(token[i]) == kept[int(float(u[i]) * len(kept))]


def test_min_p_of_one_at_an_infinite_temperature():
    """exp((l - M) / T) is 1 for every finite logit there, and 1 >= 1."""
    l = torch.randn(2, 500, generator=torch.Generator().manual_seed(1))
    l[0, ::4] = -float("inf")
    for f in (dict(), dict(k=40), dict(p=0.5)):
        _check(l, torch.tensor([0.3, 0.8]), T=float("inf"), mp=1.0, **f)
