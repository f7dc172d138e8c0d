"""ds4moe_probe's output address: the prefill plan's epilogue stores 32 bytes at a
time, so an out that begins between is refused before anything is launched."""
import pytest
import torch

import bit_quantized_moe_softmax_b200 as m
from bit_quantized_moe_softmax_b200 import synth
from tests._util import pack_with_oracle

pytestmark = pytest.mark.gpu


def test_out_between_32_bytes(orc):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()
    L = synth.float_layer(synth.TINY, 0)
    L.update(pack_with_oracle(orc, L))
    lay = m.MoELayer(256, 128, 8, 2, 64)
    lay.load(L)
    g = torch.Generator(device="cuda").manual_seed(1)
    for plan, dtype in ((0, torch.float32), (1, torch.bfloat16)):
        for which, K, N in ((0, 256, 256), (2, 128, 256)):
            x = torch.randn(4, K, generator=g, device="cuda").to(dtype)
            want = torch.empty(4, N, device="cuda")
            m.ds4moe_probe(lay.h, plan, which, 3, x, want)
            for first in (4, 8, 12, 16):   # 16 to 64 bytes
                flat = torch.full((first + 4 * N + 16,), 7.0, device="cuda")
                out = flat[first:first + 4 * N].view(4, N)
                if plan == 1 and first % 8:
                    with pytest.raises(m.Ds4MoeError) as e:
                        m.ds4moe_probe(lay.h, plan, which, 3, x, out)
                    assert e.value.status == -2 and bool((flat == 7).all())   # DS4MOE_ERR_ALIGN
                else:
                    m.ds4moe_probe(lay.h, plan, which, 3, x, out)
                    assert torch.equal(out, want) and bool((flat[:first] == 7).all()) and bool((flat[first + 4 * N:] == 7).all())
