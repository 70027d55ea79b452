"""Refusals of the LM-head's gradient entry points (no GPU: nothing launches a kernel)."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk


class FakeTensor:
    """A pointer and a size, as the binding reads them."""

    def __init__(self, ptr, nbytes=1 << 40):
        self.ptr, self.nbytes = ptr, nbytes

    def data_ptr(self):
        return self.ptr

    def numel(self):
        return self.nbytes

    def element_size(self):
        return 1


class NoStream:
    cuda_stream = 0


A = FakeTensor(0x10000000)
ODD = FakeTensor(0x10000004)
WS = FakeTensor(0x20000000)


def desc(**kw):
    base = dict(num_tokens=8, real_vocab=1000, padded_vocab=1024, ld_logits=1024,
                num_vocab_tiles=4)
    return rlk.make_desc(**{**base, **kw})


def call(d=None, k=64, h=A, w=A, tgt=A, mask=None, lse=A, g=A, gl=None, dh=A, dw=A, ws=WS):
    rlk.rlk_logp_fused_lmhead_bwd(desc() if d is None else d, h, w, k, tgt, mask, lse, g, gl, dh,
                                  dw, ws, stream=NoStream())


@pytest.mark.parametrize("kw, code", [
    (dict(k=96), rlk.RLK_ERR_BAD_SHAPE),
    (dict(k=0), rlk.RLK_ERR_BAD_SHAPE),
    (dict(k=(1 << 21) + 64), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(num_tokens=-1)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(num_tokens=(1 << 21) + 1)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(real_vocab=0)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(real_vocab=1025)), rlk.RLK_ERR_BAD_SHAPE),
    # 2^28 weight rows of 64 columns: one chunk too many
    (dict(d=desc(padded_vocab=1 << 28)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(num_vocab_tiles=0)), rlk.RLK_ERR_BAD_TILING),
    (dict(d=desc(num_virtual_shards=5)), rlk.RLK_ERR_BAD_TILING),
    (dict(dh=None, dw=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(g=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(h=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(w=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(tgt=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(lse=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(ws=None), rlk.RLK_ERR_WORKSPACE),
    (dict(h=ODD), rlk.RLK_ERR_ALIGNMENT),
    (dict(w=ODD), rlk.RLK_ERR_ALIGNMENT),
    (dict(dh=ODD), rlk.RLK_ERR_ALIGNMENT),
    (dict(dw=ODD), rlk.RLK_ERR_ALIGNMENT),
    (dict(ws=FakeTensor(0x20000010)), rlk.RLK_ERR_ALIGNMENT),
    (dict(lse=FakeTensor(0x10000002)), rlk.RLK_ERR_ALIGNMENT),
    (dict(g=FakeTensor(0x10000002)), rlk.RLK_ERR_ALIGNMENT),
    (dict(d=desc(num_tokens=0), dw=ODD), rlk.RLK_ERR_ALIGNMENT),
])
def test_refused_before_anything_runs(kw, code):
    with pytest.raises(rlk.RlkError) as ei:
        call(**kw)
    assert ei.value.status == code, ei.value


def test_workspace_bytes():
    d = desc()
    f = rlk.rlk_logp_fused_lmhead_bwd_workspace_bytes
    both, only_h, only_w = f(d, 64, True, True), f(d, 64, True, False), f(d, 64, False, True)
    assert 0 < only_h < both and 0 < only_w < both
    assert f(d, 96, True, True) == 0
    for dh, dw, need in ((A, A, both), (A, None, only_h), (None, A, only_w)):
        with pytest.raises(rlk.RlkError) as ei:
            call(dh=dh, dw=dw, ws=FakeTensor(0x20000000, need - 1))
        assert ei.value.status == rlk.RLK_ERR_WORKSPACE
    # no token and no weight gradient: nothing to do
    call(d=desc(num_tokens=0), h=None, w=None, tgt=None, lse=None, g=None, dw=None, ws=None)


def test_conveniences_check_tensors():
    n, k, v = 6, 64, 300
    h, w = torch.zeros(n, k, dtype=torch.bfloat16), torch.zeros(v, k, dtype=torch.bfloat16)
    t, f = torch.zeros(n, dtype=torch.int32), torch.zeros(n)
    kw = dict(real_vocab=v)
    b = rlk.fused_lmhead_backward
    with pytest.raises(TypeError, match="at least one"):
        b(h, w, t, None, f, **kw)
    with pytest.raises(TypeError, match="grad_logp"):
        b(h, w, t, None, f, f.double(), **kw)
    with pytest.raises(TypeError, match="lse"):
        b(h, w, t, None, f.double(), f, **kw)
    with pytest.raises(ValueError, match="6 elements"):
        b(h, w, t, None, f[:5], f, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        b(h, w, t, None, f, torch.zeros(2 * n)[::2], **kw)
    with pytest.raises(ValueError, match="contiguous"):
        b(torch.zeros(n, 2 * k, dtype=torch.bfloat16)[:, :k], w, t, None, f, f, **kw)
    with pytest.raises(TypeError, match="int32"):
        b(h, w, t.long(), None, f, f, **kw)
    with pytest.raises(ValueError, match="rows"):
        b(h, w, t, None, f, f, real_vocab=v + 1)
    with pytest.raises(ValueError, match="GPU memory"):
        b(h, w, t, None, f, f, **kw)
    with pytest.raises(TypeError, match="bfloat16"):
        rlk.lmhead_selected_token_logprob(h.float(), w, t, **kw)
    with pytest.raises(ValueError, match="GPU memory"):
        rlk.lmhead_selected_token_logprob(h, w, t, **kw)
