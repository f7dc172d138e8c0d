"""ds4moe_project over the plans that its sizes lead to: single CTAs and CTA pairs,
tiles split over two to eight of the former and two to four of the latter, each
without adapters and with adapters of small and large rank, in runs and
interleaved.  Bounds as derived in test_gpu_project.py."""
import pytest
import torch

from tests.test_gpu_project import _check, _data

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_quantized_moe_softmax_b200 import build

    build.build()


# n, in, out: the plan that the sizes have on 148 SMs
PLANS = {"pairs": (2000, 1024, 4096), "pairs, few rows": (66, 1024, 32768), "pairs by two": (1024, 4096, 4096),
         "pairs by two, ragged": (700, 4096, 4099), "pairs by two, wide": (300, 8192, 8192), "pairs by three": (200, 8192, 8192),
         "pairs by four": (700, 8192, 2000), "pairs by four, few outputs": (1500, 8192, 1000), "single": (130, 1024, 12000),
         "single by two": (512, 4096, 4096), "single by four": (256, 4096, 4090), "single by eight": (70, 2048, 1001),
         "decode": (40, 512, 9000), "decode by two": (40, 8192, 8192), "decode by four": (64, 4096, 4096),
         "decode by eight": (17, 4096, 1000), "decode, pairs": (64, 1024, 20000)}


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("na, rank, ids", [(0, 0, "none"), (6, 16, "runs"), (6, 16, "mixed"), (6, 64, "mixed"), (70, 40, "mixed"),
                                           (6, 128, "runs"), (3, 128, "mixed")])
def test_plans(plan, na, rank, ids):
    _check(_data(*PLANS[plan], na, rank, ids, seed=1))


def test_widest_input():
    """65,536 input columns: as many K blocks as there can be, split pairs and single CTAs."""
    for n, fout in ((130, 8192), (70, 500), (9, 700)):
        _check(_data(n, 65536, fout, 3, 24, "mixed"))
