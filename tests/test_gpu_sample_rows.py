"""ds4moe_sample on many rows at once, where the CTAs of a row start apart from each
other, against torch on the device."""
import pytest
import torch

import bit_quantized_moe_softmax_b200 as m

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
