"""A workspace of the embedding's gradient that overlaps another argument is
refused, on the CPU. A workspace between the rows of a strided argument is not:
such a call goes on to the device, which this machine does not have."""
import pytest
import torch

import bucketed_gradient_all_amd as ddp

# addresses that no call on the CPU ever reads
GRAD, DOUT, TOKENS, WS = 1 << 40, 2 << 40, 3 << 40, 4 << 40


def _call(d, n, grad=GRAD, dout=DOUT, tokens=TOKENS, ws=WS, accumulate=True):
    """The error's code and text: a call that passes every check asks for the device, and there is none."""
    with pytest.raises(ddp.DDPError) as e:
        ddp.ddp_embedding_grad(d, dout, tokens, n, grad, accumulate, ws, ddp.ddp_embedding_grad_workspace_bytes(d, n), 0)
    return e.value.code, e.value.msg


@pytest.fixture(autouse=True)
def no_gpu():
    if torch.cuda.device_count():
        pytest.skip("the calls that are not refused would run")


@pytest.mark.parametrize("n", [5, 9000])
@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("act,grad,index", [(0, 0, 1), (1, 0, 0), (2, 1, 1)])
def test_a_workspace_over_an_argument_is_refused(n, accumulate, act, grad, index):
    V, H = 700, 256
    d = ddp.EmbeddingDesc(V, H, act_dtype=act, grad_dtype=grad, index_dtype=index)
    need = ddp.ddp_embedding_grad_workspace_bytes(d, n)
    size = {"grad": V * H * (4 if grad == 0 else 2), "dout": n * H * (4 if act == 0 else 2),
            "tokens": n * (8 if index else 4)}
    assert _call(d, n, accumulate=accumulate)[0] == ddp.DDP_ERR_HIP
    for what, bytes_ in size.items():
        elem = 8   # every argument's alignment
        for at in (WS, WS + need - elem, WS + need // 2 // elem * elem, WS - bytes_ // elem * elem + elem):
            code, msg = _call(d, n, accumulate=accumulate, **{what: at})
            assert code == ddp.DDP_ERR_INVALID and msg == f"the workspace and {what} overlap", (what, at - WS, msg)
        for at in (WS + need, WS - (bytes_ + elem - 1) // elem * elem):
            assert _call(d, n, accumulate=accumulate, **{what: at})[0] == ddp.DDP_ERR_HIP, (what, at - WS)


@pytest.mark.parametrize("gap", [1 << 20, 1 << 28])
def test_a_workspace_between_strided_rows_is_taken(gap):
    """Rows of 64 fp32 values, `gap` elements apart."""
    V, H, n = 30, 64, 7
    d = ddp.EmbeddingDesc(V, H, grad_stride=gap, act_stride=gap)
    need = ddp.ddp_embedding_grad_workspace_bytes(d, n)
    for what, rows in (("grad", V), ("dout", n)):
        for row in (0, 1, rows - 1):
            at = WS - 4 * gap * row   # the row begins where the workspace does
            code, msg = _call(d, n, **{what: at})
            assert code == ddp.DDP_ERR_INVALID and msg == f"the workspace and {what} overlap"
            assert _call(d, n, **{what: at - 4 * H})[0] == ddp.DDP_ERR_HIP        # right before it
            assert _call(d, n, **{what: at - 4 * H + 4})[0] == ddp.DDP_ERR_INVALID
            assert _call(d, n, **{what: at + need})[0] == ddp.DDP_ERR_HIP         # right behind it
            assert _call(d, n, **{what: at + need - 4})[0] == ddp.DDP_ERR_INVALID
        # past the last row
        assert _call(d, n, **{what: WS - 4 * gap * rows})[0] == ddp.DDP_ERR_HIP


def test_one_row_for_every_position():
    d = ddp.EmbeddingDesc(30, 64, act_stride=0)
    need = ddp.ddp_embedding_grad_workspace_bytes(d, 5000)
    for at, code in ((WS, ddp.DDP_ERR_INVALID), (WS - 252, ddp.DDP_ERR_INVALID), (WS - 256, ddp.DDP_ERR_HIP),
                     (WS + need - 4, ddp.DDP_ERR_INVALID), (WS + need, ddp.DDP_ERR_HIP)):
        assert _call(d, 5000, dout=at)[0] == code, at - WS
