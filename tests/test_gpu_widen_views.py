"""ds4moe_widen_rows into views: ``out`` may begin at any 16-byte address, and what
lies around it stays."""
import pytest
import torch

import bit_quantized_moe_softmax_b200 as m

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()


@pytest.mark.parametrize("start", [16, 32, 48, 4112])
@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("n, H", [(1, 8), (3, 2056), (61, 2050), (1100, 4104)])
def test_out_at_every_16_bytes(start, out_type, n, H):
    """Few rows (a piece per thread) and many (two), bytes behind a 4096-byte boundary that are no multiple of 32."""
    g = torch.Generator().manual_seed(n + H)
    q = torch.randint(-127, 128, (n, H), generator=g, dtype=torch.int8)
    scale = torch.rand(n, -(-H // 128), generator=g) + 0.5
    size = 2 if out_type == BF16 else 4
    first, count = start // size, n * H
    flat = torch.full((first + count + 64,), 9.0, dtype=out_type, device="cuda")
    assert flat.data_ptr() % 512 == 0
    view = flat[first:first + count].view(n, H)
    m.ds4moe_widen_rows(q.cuda(), scale.cuda(), view)
    torch.cuda.synchronize()
    want = (q.float() * scale.repeat_interleave(128, 1)[:, :H]).to(out_type)
    assert torch.equal(view.cpu(), want)
    assert bool((flat[:first] == 9).all()) and bool((flat[first + count:] == 9).all())
    # a row view of a contiguous buffer
    rows = torch.full((n + 1, H), 9.0, dtype=out_type, device="cuda")
    if rows[1:].data_ptr() % 16 == 0:
        m.ds4moe_widen_rows(q.cuda(), scale.cuda(), rows[1:])
        assert torch.equal(rows[1:].cpu(), want) and bool((rows[0] == 9).all())


def test_q_at_every_16_bytes():
    """The codes' reads are 16 bytes wide: a view that begins at any multiple of 16."""
    n, H = 5, 2056
    for start in (16, 32, 48):
        flat = torch.randint(-127, 128, (start + n * H,), dtype=torch.int8, device="cuda")
        q = flat[start:].view(n, H)
        out = torch.empty(n, H, dtype=BF16, device="cuda")
        m.ds4moe_widen_rows(q, torch.full((n, 1), 0.5, device="cuda"), out, group=0)
        assert torch.equal(out, (q.float() * 0.5).to(BF16))
