"""The projection's bounded waits when they run out, with no GPU fault, trap or hang.

ds4moe_selftest_project_wait runs the projection with waits that give up at
once from a given tile of each CTA on: what they kept from being computed is
NaN, whatever out held before, the error word is set, and the next call is as
if nothing had been.
"""
import ctypes

import pytest
import torch

import bit_quantized_moe_softmax_b200 as m
from tests.test_gpu_project import _data, _reference

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()


# rows, in, out, adapters, rank: single CTAs and CTA pairs, whole and split tiles, a decode batch's adapters by the
# draining warps and others as K blocks, one tile per CTA and several
FORMS = {"single": (200, 512, 4000, 0, 0), "single, adapters": (200, 512, 4000, 3, 16), "single, split": (256, 4096, 4096, 0, 0),
         "single, split, adapters": (100, 2048, 4000, 5, 40), "decode": (40, 512, 9000, 3, 16), "decode, split": (64, 4096, 4096, 4, 32),
         "pairs": (2000, 1024, 4096, 0, 0), "pairs, adapters": (1030, 264, 10007, 6, 48), "pairs, split": (700, 4096, 4096, 0, 0),
         "pairs, split, adapters": (300, 8192, 8192, 4, 16), "pairs, decode": (64, 1024, 20000, 4, 16),
         "several tiles": (90, 512, 40000, 0, 0), "several tiles, decode": (30, 512, 40000, 3, 24),
         "several tiles, pairs": (3000, 512, 9000, 2, 8)}


def _error():
    code = ctypes.c_int32(0)
    return m.lib().ds4moe_get_project_error(torch.cuda.current_stream().cuda_stream, ctypes.byref(code)), code.value


@pytest.mark.parametrize("form", FORMS)
def test_waits_that_give_up_at_once(form):
    n, fin, fout, na, rank = FORMS[form]
    d = _data(n, fin, fout, na, rank, "runs")
    want = torch.empty(n, fout, dtype=BF16, device="cuda")
    m.ds4moe_project(out=want, **d)
    for _ in range(2):
        out = torch.full((n + 1, fout), 3.0, dtype=BF16, device="cuda")
        m.ds4moe_selftest_project_wait(out=out[:n], **d)
        assert _error() == (-6, 2)   # DS4MOE_ERR_TIMEOUT, bit 1
        assert bool(out[:n].isnan().all()) and bool((out[n] == 3).all())
        assert _error() == (0, 0)    # read and cleared
        m.ds4moe_project(out=out[:n], **d)
        assert torch.equal(out[:n], want) and _error() == (0, 0)


@pytest.mark.parametrize("form", ["several tiles", "several tiles, decode", "several tiles, pairs"])
@pytest.mark.parametrize("tiles", [1, 2])
def test_later_tiles_give_up(form, tiles):
    """From the second (or third) tile of a CTA on: those are NaN, the earlier ones NaN or right."""
    n, fin, fout, na, rank = FORMS[form]
    d = _data(n, fin, fout, na, rank, "runs")
    y, bound = _reference(d)
    for _ in range(4):
        out = torch.full((n, fout), 3.0, dtype=BF16, device="cuda")
        m.ds4moe_selftest_project_wait(out=out, tiles=tiles, **d)
        status = _error()
        nan = out.isnan()
        assert bool((nan | ((out.double() - y).abs() <= bound)).all())
        assert status in ((-6, 2), (0, 0)) and bool(nan.any()) == (status != (0, 0))
        if n <= 90:   # one tile along the rows, of 128 outputs each
            later = torch.cuda.get_device_properties(0).multi_processor_count * tiles * 128
            assert later < fout and bool(nan[:, later:].all()) and status == (-6, 2)
        m.ds4moe_project(out=out, **d)
        assert bool(((out.double() - y).abs() <= bound).all()) and _error() == (0, 0)


def test_no_wait_gives_up_in_time():
    """With more tiles in time than a CTA has, it is the projection."""
    d = _data(90, 512, 40000, 3, 16, "runs")
    a, b = (torch.empty(90, 40000, dtype=BF16, device="cuda") for _ in range(2))
    m.ds4moe_project(out=a, **d)
    m.ds4moe_selftest_project_wait(out=b, tiles=1000, **d)
    assert torch.equal(a, b) and _error() == (0, 0)


def test_error_word_is_taken_in_one_step():
    """Reads on one stream while projections that give up run on another: every error is in some answer."""
    d = _data(8, 512, 640, 0, 0)
    out = torch.empty(8, 640, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = 0
    for _ in range(50):
        m.ds4moe_selftest_project_wait(out=out, stream=side, **d)
        seen += _error()[1] == 2
        side.synchronize()
        seen += _error()[1] == 2
        assert seen >= 1
        seen = 0
