"""The AdamW step's binding on the CPU: what its defaults hand to the library."""
import ctypes
import math
import types

import bucketed_gradient_all_amd as ddp


def _given(**kw):
    """The ddp_adamw_args that a call hands over."""
    seen = []

    def step(handle, args, stream):
        seen.append(ddp.ddp_adamw_args.from_buffer_copy(ctypes.cast(args, ctypes.POINTER(ddp.ddp_adamw_args)).contents))
        return ddp.DDP_OK

    o = ddp.AdamW(0)
    o._lib = types.SimpleNamespace(ddp_adamw_step=step)
    ddp.ddp_adamw_step(o, 1e-3, 7, 0, **kw)
    return seen[0]


def test_a_norm_without_a_bound_does_not_clip():
    """A bound of 0 would leave nothing of the gradients."""
    a = _given(norm=0x1000, skip_nonfinite=True)
    assert a.norm == 0x1000 and a.skip_nonfinite == 1 and a.max_norm == math.inf


def test_arguments_reach_their_fields():
    a = _given(beta1=0.8, beta2=0.95, eps=1e-6, max_norm=2.0, norm=0x1000, lr_ptr=0x2000, step_ptr=0x3000)
    assert (a.lr, a.step, a.beta1, a.beta2, a.eps, a.max_norm) == (1e-3, 7, 0.8, 0.95, 1e-6, 2.0)
    assert (a.norm, a.lr_ptr, a.step_ptr, a.skip_nonfinite) == (0x1000, 0x2000, 0x3000, 0)
    b = _given()
    assert b.norm is None and b.lr_ptr is None and b.step_ptr is None and (b.beta1, b.beta2, b.eps) == (0.9, 0.999, 1e-8)
