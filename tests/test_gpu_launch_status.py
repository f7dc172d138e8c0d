"""An error that an earlier call left behind is not the next launch's: the operators
around the layer report their own launch, and launch once."""
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


def _leave_an_error_behind():
    """The library refuses to synchronize with a stream under capture: a CUDA error of the host call alone."""
    from cuda.bindings import runtime as rt

    st = torch.cuda.Stream()
    assert rt.cudaStreamBeginCapture(st.cuda_stream, rt.cudaStreamCaptureMode.cudaStreamCaptureModeThreadLocal)[0] == 0
    with pytest.raises(m.Ds4MoeError) as e:
        m.ds4moe_get_project_error(st)
    rt.cudaStreamEndCapture(st.cuda_stream)
    rt.cudaGetLastError()
    assert e.value.status == -5


@pytest.mark.parametrize("stream", [None, "explicit"])
def test_norm_in_place_and_widening_launch_once(stream):
    st = None if stream is None else torch.cuda.current_stream()
    x, total, w = torch.ones(3, 64, device="cuda"), torch.full((3, 64), 5.0, device="cuda"), torch.ones(64, device="cuda")
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    _leave_an_error_behind()
    m.ds4moe_add_rmsnorm(x, w, 1e-6, residual=total, sum=total, out=out, stream=st)
    assert bool((total == 6).all())
    _leave_an_error_behind()
    m.ds4moe_widen_rows(torch.ones(3, 64, dtype=torch.int8, device="cuda"), torch.ones(3, 1, device="cuda"), out, stream=st)
    assert bool((out == 1).all())
    _leave_an_error_behind()
    u, token = torch.zeros(3, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    m.ds4moe_sample(total, u, token, stream=st)
    assert token.tolist() == [0, 0, 0]
    _leave_an_error_behind()
    b = x.bfloat16()
    y = torch.empty(3, 3, dtype=torch.bfloat16, device="cuda")
    m.ds4moe_project(b, b.clone(), y, stream=st)
    assert bool((y == 64).all())
