"""A CUDA error is reported by the call that met it, and by no call after it.

The error here is the runtime's refusal, on the host, to wait for a stream that is being captured
into a graph: nothing is launched."""
import ctypes

import pytest
import torch

from test_gpu_train import check_loss, run_loss

pytestmark = pytest.mark.gpu

RELAXED = 2


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["full", "bias", "d2t"])
def test_an_error_is_not_reported_again(form, dtype):
    from dspark_block_drafter_gb300 import DSparkError, _abi
    from dspark_block_drafter_gb300 import torch_io as tio
    out, o, args = run_loss(40, 64, 512, 8, dtype, form=form, n_emit=104)
    ws = args[6]
    driver = ctypes.CDLL("libcuda.so.1")
    s = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert driver.cuStreamBeginCapture_v2(handle, RELAXED) == 0
    status = tio.device_status(ws, stream=s)
    assert driver.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0      # (now invalid)
    assert status == _abi.DSPARK_ERR_CUDA and not graph.value
    for f in (out.loss, out.d_hidden, out.d_lm_head):
        f.fill_(float("nan"))
    try:
        tio.head_loss(*args)
    except DSparkError as e:
        pytest.fail(f"an earlier call's error: {e}")
    torch.cuda.synchronize()
    assert tio.device_status(ws) == 0
    check_loss(out, o, dtype)
