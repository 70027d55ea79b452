"""The LM-head's gradients where inputs are not ordinary numbers or not there at all.  Needs an
MI355X."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import lmhead_cases as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def bits(t):
    return t.contiguous().view(torch.int16)


def make(n, k, v, pad, seed):
    c = C.make_case(n, k, v, pad, seed, DEV, mask_keep=1.0, ignore_frac=0.0)
    _, lse = rlk.fused_lmhead(c.h, c.w, c.tgt, c.mask, real_vocab=v, num_vocab_tiles=1)
    return c, lse


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("terms", ["logp", "lse"])
@pytest.mark.parametrize("n", [20, 300])
def test_lse_that_is_not_finite(n, terms, value):
    """It has no probabilities: NaN for its row of dhidden and for every real row of dweight;
    the other rows of dhidden keep their bits, the padding of dweight its zeros."""
    print(f"case n {n} {terms} {value}", flush=True)
    c, lse = make(n, 64, 600, 640, n)
    g, gl = (c.g, None) if terms == "logp" else (None, c.gl)
    top = int((c.g if terms == "logp" else c.gl).abs().argmax())
    row = (top + 1) % n
    ref, _ = rlk.fused_lmhead_backward(c.h, c.w, c.tgt, None, lse, g, gl, real_vocab=600)
    lse[row] = value
    dh, dw = rlk.fused_lmhead_backward(c.h, c.w, c.tgt, None, lse, g, gl, real_vocab=600,
                                       validate=True)  # no data error
    rest = torch.arange(n, device=DEV) != row
    assert dh[row].isnan().all() and torch.equal(bits(dh[rest]), bits(ref[rest]))
    assert dw[:600].isnan().all() and (bits(dw[600:]) == 0).all()
    # a row that no term reaches may hold it
    if g is not None:
        c.mask[row] = False
        dh, dw = rlk.fused_lmhead_backward(c.h, c.w, c.tgt, c.mask, lse, g, None, real_vocab=600)
        assert (bits(dh[row]) == 0).all() and dw.float().isfinite().all()


def test_no_token_and_a_frozen_head():
    c, lse = make(5, 64, 300, 300, 8)
    h = c.h[:0].clone().requires_grad_(True)
    logp, out = rlk.lmhead_selected_token_logprob(h, c.w, c.tgt[:0], None, real_vocab=300,
                                                  num_vocab_tiles=1)
    (logp.sum() + out.sum()).backward()
    assert h.grad.shape == (0, 64)
    dh, dw = rlk.fused_lmhead_backward(c.h[:0], c.w, c.tgt[:0], None, lse[:0], c.g[:0],
                                       real_vocab=300, want_weight=False)
    assert dh.shape == (0, 64) and dw is None
