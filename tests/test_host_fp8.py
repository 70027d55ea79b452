"""Refusals of the 8-bit LM-head's entry points (no GPU: nothing launches a kernel)."""
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
PTR = 0x10000000


def desc(**kw):
    base = dict(num_tokens=8, real_vocab=1000, padded_vocab=1024, ld_logits=1024,
                num_vocab_tiles=4)
    return rlk.make_desc(**{**base, **kw})


def matrix(q=PTR, scale=PTR, rs=1, cs=8):
    return rlk.rlk_fp8_matrix(q, scale, rs, cs)


def fused(d=None, h=matrix(), w=matrix(), k=128, tgt=A, logp=A, lse=A, ws=FakeTensor(0x20000000)):
    rlk.rlk_logp_fused_lmhead_fp8(desc() if d is None else d, h, w, k, tgt, None, logp, lse, ws,
                                  stream=NoStream())


def logits(d=None, h=matrix(), w=matrix(), k=128, out=A):
    rlk.rlk_lmhead_logits_fp8(desc() if d is None else d, h, w, k, out, stream=NoStream())


def quantize(rows=8, cols=128, x=A, ld=128, block_rows=1, q=A, scale=A, rs=1, cs=8):
    rlk.rlk_fp8_quantize(rows, cols, x, ld, block_rows, q, scale, rs, cs, stream=NoStream())


def refused(call, code, **kw):
    with pytest.raises(rlk.RlkError) as ei:
        call(**kw)
    assert ei.value.status == code, ei.value


@pytest.mark.parametrize("call", [fused, logits])
@pytest.mark.parametrize("kw, code", [
    (dict(k=64), rlk.RLK_ERR_BAD_SHAPE),
    (dict(k=192), rlk.RLK_ERR_BAD_SHAPE),
    (dict(k=0), rlk.RLK_ERR_BAD_SHAPE),
    (dict(k=(1 << 21) + 128), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(num_tokens=-1)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(real_vocab=1025)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(num_vocab_tiles=0)), rlk.RLK_ERR_BAD_TILING),
    (dict(h=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(w=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(h=matrix(q=None)), rlk.RLK_ERR_NULL_POINTER),
    (dict(w=matrix(scale=None)), rlk.RLK_ERR_NULL_POINTER),
    (dict(h=matrix(q=PTR + 8)), rlk.RLK_ERR_ALIGNMENT),
    (dict(w=matrix(scale=PTR + 2)), rlk.RLK_ERR_ALIGNMENT),
    (dict(h=matrix(rs=0)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(w=matrix(cs=-1)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(h=matrix(rs=1 << 22)), rlk.RLK_ERR_BAD_SHAPE),  # 256 tokens' scales span 2^32 bytes
    # 2^28 tokens of 128 columns: one chunk too many
    (dict(d=desc(num_tokens=1 << 28)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(real_vocab=1 << 28, padded_vocab=1 << 28, ld_logits=1 << 28)),
     rlk.RLK_ERR_BAD_SHAPE),
])
def test_products_refuse(call, kw, code):
    refused(call, code, **kw)


def test_fused_refuses():
    refused(fused, rlk.RLK_ERR_BAD_TILING, d=desc(num_vocab_tiles=5))  # tiles under 256 columns
    refused(fused, rlk.RLK_ERR_NULL_POINTER, tgt=None)
    refused(fused, rlk.RLK_ERR_NULL_POINTER, lse=None)
    refused(fused, rlk.RLK_ERR_WORKSPACE, ws=None)
    need = rlk.rlk_logp_fused_lmhead_fp8_workspace_bytes(desc())
    # z of 8 tokens x 1000 columns, rounded up to 1024, beside the bf16 head's workspace
    assert need == rlk.rlk_logp_fused_lmhead_workspace_bytes(desc()) + 8 * 1024 * 4
    many = desc(num_tokens=65)
    assert rlk.rlk_logp_fused_lmhead_fp8_workspace_bytes(many) == \
        rlk.rlk_logp_fused_lmhead_workspace_bytes(many)
    refused(fused, rlk.RLK_ERR_WORKSPACE, ws=FakeTensor(0x20000000, need - 1))
    refused(fused, rlk.RLK_ERR_ALIGNMENT, ws=FakeTensor(0x20000010))
    fused(d=desc(num_tokens=0), h=None, w=None, tgt=None, logp=None, lse=None, ws=None)


def test_logits_refuse():
    refused(logits, rlk.RLK_ERR_NULL_POINTER, out=None)
    refused(logits, rlk.RLK_ERR_ALIGNMENT, out=FakeTensor(PTR + 8))
    refused(logits, rlk.RLK_ERR_BAD_SHAPE, d=desc(ld_logits=1016))
    refused(logits, rlk.RLK_ERR_ALIGNMENT, d=desc(ld_logits=1028))
    refused(logits, rlk.RLK_ERR_BAD_SHAPE, d=desc(validate=True))
    # column numbers of the last block would pass 2^31
    refused(logits, rlk.RLK_ERR_BAD_SHAPE, d=desc(padded_vocab=(1 << 31) - 256,
                                                  ld_logits=(1 << 31) - 256))
    logits(d=desc(num_tokens=0), h=None, w=None, out=None)


@pytest.mark.parametrize("kw, code", [
    (dict(rows=-1), rlk.RLK_ERR_BAD_SHAPE),
    (dict(cols=64), rlk.RLK_ERR_BAD_SHAPE),
    (dict(cols=200, ld=200), rlk.RLK_ERR_BAD_SHAPE),
    (dict(block_rows=2), rlk.RLK_ERR_BAD_TILING),
    (dict(ld=120), rlk.RLK_ERR_BAD_SHAPE),
    (dict(ld=132), rlk.RLK_ERR_ALIGNMENT),
    (dict(rs=0), rlk.RLK_ERR_BAD_SHAPE),
    (dict(cs=0), rlk.RLK_ERR_BAD_SHAPE),
    (dict(x=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(q=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(scale=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(x=FakeTensor(PTR + 8)), rlk.RLK_ERR_ALIGNMENT),
    (dict(q=FakeTensor(PTR + 8)), rlk.RLK_ERR_ALIGNMENT),
])
def test_quantize_refuses(kw, code):
    refused(quantize, code, **kw)
    quantize(rows=0, x=None, q=None, scale=None)


def test_conveniences_check_tensors():
    n, k, v = 6, 256, 300
    x = torch.zeros(n, k, dtype=torch.bfloat16)
    hq, hs = torch.zeros(n, k).to(torch.float8_e4m3fn), torch.ones(n, 2)
    wq, ws = torch.zeros(v, k).to(torch.float8_e4m3fn), torch.ones(3, 2)
    t = torch.zeros(n, dtype=torch.int32)
    with pytest.raises(TypeError, match="bfloat16"):
        rlk.quantize_fp8(x.float())
    with pytest.raises(ValueError, match="block_rows"):
        rlk.quantize_fp8(x, 64)
    with pytest.raises(ValueError, match="128 columns"):
        rlk.quantize_fp8(x[:, :130])
    with pytest.raises(ValueError, match="GPU memory"):
        rlk.quantize_fp8(x)
    for call in (lambda *a, **kw: rlk.lmhead_logits_fp8(*a, real_vocab=v, **kw),
                 lambda *a, **kw: rlk.fused_lmhead_fp8(*a, t, real_vocab=v, num_vocab_tiles=1,
                                                       **kw)):
        with pytest.raises(TypeError, match="float8"):
            call(x, wq.float(), ws)
        with pytest.raises(TypeError, match="float32"):
            call(x, wq, ws.double())
        with pytest.raises(ValueError, match="shape"):
            call(x, wq, ws[:2])
        with pytest.raises(ValueError, match="shape"):
            call((hq, hs.t()), wq, ws)
        with pytest.raises(ValueError, match="positive strides"):
            call((hq, torch.ones(1, 2).expand(n, 2)), wq, ws)
        with pytest.raises(TypeError, match="bfloat16"):
            call(x.float(), wq, ws)
        with pytest.raises(ValueError, match="columns"):
            call(x[:, :128].contiguous(), wq, ws)
        with pytest.raises(ValueError, match="contiguous"):
            call((hq.t().contiguous().t(), hs), wq, ws)
        with pytest.raises(ValueError, match="GPU memory"):
            call(x, wq, ws)
        with pytest.raises(ValueError, match="GPU memory"):
            call((hq, hs), wq, ws)
    with pytest.raises(ValueError, match="rows"):
        rlk.lmhead_logits_fp8(x, wq, ws, real_vocab=v + 1)
    with pytest.raises(TypeError, match="int32"):
        rlk.fused_lmhead_fp8(x, wq, ws, t.long(), real_vocab=v)
