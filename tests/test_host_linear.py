"""Refusals of the dense products' entry points, and the slopes that their GPU tests are held to
against differences (no GPU: nothing launches a kernel)."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import linear_cases as C
from tests.test_host_fp8 import FakeTensor, NoStream, refused

X, W, OUT, WS = (FakeTensor(p) for p in (0x10000000, 0x18000000, 0x20000000, 0x30000000))
PTR = 0x40000000


def desc(**kw):
    d = dict(tokens=8, in_dim=128, out_dim=100, padded_out=104, ld_out=104, ld_residual=100,
             ld_saved=104, activation=rlk.ACTIVATIONS["silu"], bias_dtype=rlk.RLK_DTYPE_F32,
             saved_dtype=rlk.RLK_DTYPE_F16, cap=0.0)
    return rlk.rlk_linear_desc(**{**d, **kw})


def forward(d=None, x=X, w=W, bias=None, residual=None, out=OUT, saved=None):
    rlk.rlk_linear_fwd(desc() if d is None else d, x, w, bias, residual, out, saved,
                       stream=NoStream())


def backward(d=None, x=X, w=W, saved=X, dy=X, ld=100, dx=OUT, dw=OUT, db=OUT, ws=WS):
    rlk.rlk_linear_bwd(desc() if d is None else d, x, w, saved, dy, ld, dx, dw, db, ws,
                       stream=NoStream())


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw, code", [
    (dict(d=desc(tokens=-1)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(tokens=(1 << 31) - 1)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(in_dim=96)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(in_dim=0)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(in_dim=(1 << 21) + 64)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(out_dim=0)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(out_dim=(1 << 31) - 8)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(activation=6)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(activation=-1)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(activation=5, cap=0.0)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(activation=5, cap=float("nan"))), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(activation=5, cap=float("inf"))), rlk.RLK_ERR_BAD_SHAPE),
    (dict(x=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(w=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(x=FakeTensor(PTR + 8)), rlk.RLK_ERR_ALIGNMENT),
    (dict(w=FakeTensor(PTR + 2)), rlk.RLK_ERR_ALIGNMENT),
    (dict(saved=X, d=desc(ld_saved=96)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(saved=X, d=desc(ld_saved=108)), rlk.RLK_ERR_ALIGNMENT),
    (dict(saved=FakeTensor(PTR + 8)), rlk.RLK_ERR_ALIGNMENT),
    (dict(saved=X, d=desc(saved_dtype=rlk.RLK_DTYPE_BF16)), rlk.RLK_ERR_DTYPE),
])
def test_calls_refuse(call, kw, code):
    refused(call, code, **kw)


def test_forward_refuses():
    refused(forward, rlk.RLK_ERR_BAD_SHAPE, d=desc(padded_out=99))
    refused(forward, rlk.RLK_ERR_BAD_SHAPE, d=desc(ld_out=96))
    refused(forward, rlk.RLK_ERR_ALIGNMENT, d=desc(ld_out=108))
    refused(forward, rlk.RLK_ERR_BAD_SHAPE, residual=X, d=desc(ld_residual=99))
    refused(forward, rlk.RLK_ERR_ALIGNMENT, residual=FakeTensor(PTR + 1))
    refused(forward, rlk.RLK_ERR_BAD_SHAPE, residual=OUT)
    refused(forward, rlk.RLK_ERR_NULL_POINTER, out=None)
    refused(forward, rlk.RLK_ERR_ALIGNMENT, out=FakeTensor(PTR + 8))
    refused(forward, rlk.RLK_ERR_DTYPE, bias=X, d=desc(bias_dtype=2))
    refused(forward, rlk.RLK_ERR_ALIGNMENT, bias=FakeTensor(PTR + 2))
    forward(d=desc(tokens=0), x=None, w=None, out=None)


def test_backward_refuses():
    refused(backward, rlk.RLK_ERR_BAD_SHAPE, d=desc(out_dim=(1 << 21) + 1, ld_saved=1 << 22),
            ld=1 << 22)
    refused(backward, rlk.RLK_ERR_BAD_SHAPE, ld=99)
    refused(backward, rlk.RLK_ERR_NULL_POINTER, dy=None)
    refused(backward, rlk.RLK_ERR_NULL_POINTER, saved=None)
    refused(backward, rlk.RLK_ERR_NULL_POINTER, dx=None, dw=None, db=None)
    refused(backward, rlk.RLK_ERR_ALIGNMENT, dx=FakeTensor(PTR + 8))
    refused(backward, rlk.RLK_ERR_ALIGNMENT, db=FakeTensor(PTR + 2))
    refused(backward, rlk.RLK_ERR_DTYPE, d=desc(bias_dtype=3))
    refused(backward, rlk.RLK_ERR_WORKSPACE, ws=None)
    refused(backward, rlk.RLK_ERR_ALIGNMENT, ws=FakeTensor(PTR + 16))
    need = rlk.rlk_linear_bwd_workspace_bytes(desc())
    assert need > 0
    refused(backward, rlk.RLK_ERR_WORKSPACE, ws=FakeTensor(0x30000000, need - 1))
    assert rlk.rlk_linear_bwd_workspace_bytes(desc(in_dim=1)) == 0


def test_outputs_stand_apart():
    """An output that is an input, or another output, would be written while it is read."""
    a, b, c, e = (FakeTensor(PTR + i * 0x1000000) for i in range(4))
    for kw in (dict(out=X), dict(out=W), dict(out=OUT, saved=OUT), dict(saved=X), dict(saved=W),
               dict(residual=a, saved=a), dict(bias=a, out=a), dict(bias=a, saved=a)):
        refused(forward, rlk.RLK_ERR_BAD_SHAPE, **kw)
    ws = FakeTensor(0x30000000, 1 << 20)
    apart = dict(saved=a, dy=b, dx=c, dw=e, db=None, ws=ws)
    for kw in (dict(dx=X), dict(dx=W), dict(dx=a), dict(dx=b), dict(dw=X), dict(dw=W),
               dict(dw=a), dict(dw=b), dict(dw=c), dict(db=c), dict(db=e), dict(db=W),
               dict(dx=ws), dict(dy=ws), dict(saved=ws)):
        refused(backward, rlk.RLK_ERR_BAD_SHAPE, **{**apart, **kw})


@pytest.mark.parametrize("cap", [1e-39, 9e-31, 2e30, 3e38])
def test_caps_whose_quotients_leave_fp32_are_refused(cap):
    refused(forward, rlk.RLK_ERR_BAD_SHAPE, d=desc(activation=5, cap=cap))
    refused(backward, rlk.RLK_ERR_BAD_SHAPE, d=desc(activation=5, cap=cap))
    x = torch.zeros(5, 64, dtype=torch.bfloat16)
    for call in (rlk.linear_forward, rlk.head_linear):
        with pytest.raises(ValueError, match="cap must"):
            call(x, x, activation="softcap", cap=cap)
    with pytest.raises(ValueError, match="cap must"):
        rlk.lmhead_logits(x, x, cap=cap, real_vocab=5)


def test_conveniences_check_tensors():
    bf = dict(dtype=torch.bfloat16)
    x, w, b = torch.zeros(5, 64, **bf), torch.zeros(9, 64, **bf), torch.zeros(9)
    r = torch.zeros(5, 9, **bf)
    for call in (rlk.linear_forward, rlk.head_linear):
        with pytest.raises(ValueError, match="activation"):
            call(x, w, activation="swish")
        with pytest.raises(ValueError, match="cap goes"):
            call(x, w, activation="softcap")
        with pytest.raises(ValueError, match="cap goes"):
            call(x, w, activation="relu", cap=1.0)
        with pytest.raises(ValueError, match="finite"):
            call(x, w, activation="softcap", cap=-1.0)
        with pytest.raises(TypeError, match="bfloat16"):
            call(x.float(), w)
        with pytest.raises(TypeError, match="bfloat16"):
            call(x, w, residual=r.float())
        with pytest.raises(ValueError, match="contiguous"):
            call(torch.zeros(5, 128, **bf)[:, :64], w)
        with pytest.raises(ValueError, match="columns"):
            call(x, torch.zeros(9, 128, **bf))
        with pytest.raises(TypeError, match="bias"):
            call(x, w, b.double())
        with pytest.raises(ValueError, match="bias"):
            call(x, w, b[:8])
        with pytest.raises(ValueError, match="shape"):
            call(x, w, b, r[:, :8])
        with pytest.raises(ValueError, match="GPU memory"):
            call(x, w, b, r)
    for kw in (dict(want_x=False, want_weight=False), dict(bias_dtype=torch.float16)):
        with pytest.raises(ValueError, match="want_|bias_dtype"):
            rlk.linear_backward(x, w, r, **kw)
    with pytest.raises(TypeError, match="grad_out"):
        rlk.linear_backward(x, w, None)
    with pytest.raises(ValueError, match="rows, fewer"):
        rlk.lmhead_logits(x, w, real_vocab=10)
    with pytest.raises(ValueError, match="GPU memory"):
        rlk.lmhead_logits(x, w, b, real_vocab=9)


@pytest.mark.parametrize("act", C.ACTS)
def test_slopes_against_differences(act):
    """Central differences with a step of 2^-12: the third derivatives stay below 4, so they are
    off by less than 4/6 2^-24 and the roundings of the difference, 2^-52 2^12 8."""
    z = torch.linspace(-9, 9, 4001, dtype=torch.float64) + 2.0 ** -10  # (off relu's corner)
    s = 2.0 ** -12
    got = (C.act64(z + s, act) - C.act64(z - s, act)) / (2 * s)
    assert (got - C.slope64(z, act)).abs().max() < 4 / 6 * 2.0 ** -24 + 2.0 ** -37
