"""GPU: a list whose workspace and scratch lie at the least alignment that the
header asks for, 16 and 8 bytes."""
import pytest

from test_gpu_grads import Case, _lib, _torch, check_clip, check_norm, new_norm, ref_norm, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("numel", [[5, 0, 8191], [300000, 17, 64] * 9])
@pytest.mark.parametrize("apart", [False, True])
def test_the_least_alignment(numel, apart):
    torch, ddp = _torch(), _lib()
    say("case alignment", len(numel), apart)
    c = Case(numel, copies=2, out=[0] * len(numel) if apart else None, seed=3)
    out = [[v.data_ptr() for v in vs] for vs in c.out_views] if apart else None
    desc = ddp.GradsDesc(numel, [[v.data_ptr() for v in vs] for vs in c.views], c.dtype, out, c.out_dtype)
    need = ddp.ddp_grads_workspace_bytes(desc)
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    desc.set_workspace(ws.data_ptr() + 16, need)
    g = ddp.ddp_grads_create(desc)
    n = ddp.ddp_grads_scratch_bytes(g)
    scratch = torch.full((n + 16,), 0xAB, dtype=torch.uint8, device="cuda")
    norm = new_norm()
    ddp.ddp_clip_grad_norm(g, 2, 0.5, norm.data_ptr(), torch.cuda.current_stream().cuda_stream,
                           scratch.data_ptr() + 8, n)
    want = ref_norm(c.flat64(), 2)
    check_norm(float(norm), want)
    check_clip(c, want, 0.5)
    c.guards_hold()
    for buf, lo, hi in ((ws, 16, 16 + need), (scratch, 8, 8 + n)):
        assert bool((buf[:lo] == 0xAB).all()) and bool((buf[hi:] == 0xAB).all())
    ddp.ddp_grads_destroy(g)
