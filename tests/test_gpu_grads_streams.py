"""GPU: lists of gradients and the streams their calls were queued on."""
import ctypes

import pytest

from test_gpu_grads import Case, _lib, _torch, check_clip, check_norm, new_norm, ref_norm, say

pytestmark = pytest.mark.gpu


def _stream_of_ones_own():
    """A stream that torch knows nothing of, at the default priority."""
    hip = ctypes.CDLL("libamdhip64.so")
    hip.hipStreamDestroy.argtypes = [ctypes.c_void_p]
    s = ctypes.c_void_p()
    assert hip.hipStreamCreate(ctypes.byref(s)) == 0
    return hip, s.value


@pytest.mark.parametrize("destroy", [False, True])
def test_a_list_outlives_the_stream_it_was_used_on(destroy):
    torch, ddp = _torch(), _lib()
    say("case stream gone", destroy)
    hip, s = _stream_of_ones_own()
    c = Case([300000, 17], out=[0, 1], seed=31)
    norm = new_norm()
    torch.cuda.synchronize()
    g = c.make()
    ddp.ddp_clip_grad_norm(g, 2, 0.5, norm.data_ptr(), s)
    assert hip.hipStreamSynchronize(ctypes.c_void_p(s)) == 0
    assert hip.hipStreamDestroy(s) == 0
    if destroy:
        ddp.ddp_grads_destroy(g)
    held = [g.workspace.data_ptr(), g.scratch.data_ptr()]
    del g
    assert {t.data_ptr() for t in ddp._parked} >= set(held)
    want = ref_norm(c.flat64(), 2)
    check_norm(float(norm), want)
    check_clip(c, want, 0.5)
    g = c.make()   # drains the device and frees what was parked
    assert ddp._parked == []
    norm.fill_(-1.0)
    ddp.ddp_grad_norm(g, 2, norm.data_ptr(), torch.cuda.current_stream().cuda_stream)
    check_norm(float(norm), want)
