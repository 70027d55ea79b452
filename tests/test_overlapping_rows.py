"""What the logit rules' calls write may not lie across the logits that they read: another block could
still read there.  Rows beside the logits' own, in one buffer, are fine."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import process_cases as C
from tests.test_host_fp8 import FakeTensor, refused
from tests.test_host_process import backward, desc, process

BF16, F32 = rlk.RLK_DTYPE_BF16, rlk.RLK_DTYPE_F32
PTR = 0x10000000
LOGITS = FakeTensor(PTR)


@pytest.mark.parametrize("call", [process, backward])
@pytest.mark.parametrize("at, ld, dtype", [
    (16, 1024, BF16),               # the same rows, 8 columns on
    (-16, 1024, BF16),
    (2048, 1024, BF16),             # a row on
    (-2048, 1024, BF16),
    (7 * 2048 + 1984, 1024, BF16),  # its first row begins in the logits' last one
    (-2032 - 7 * 2048, 1024, BF16),
    (4096, 2048, BF16),             # other strides
    (-16, 1024, F32),
    (7 * 2048 + 1984, 1024, F32),
    (16, 1 << 62, BF16),            # a stride whose bytes pass 64 bits
])
def test_overlaps_are_refused(call, at, ld, dtype):
    refused(call, rlk.RLK_ERR_BAD_SHAPE, x=LOGITS, out=FakeTensor(PTR + at), ld=ld, dtype=dtype)


@pytest.mark.parametrize("call", [process, backward])
@pytest.mark.parametrize("at", [1984, 8192 + 1984, -64, -8192 - 64])
def test_overlaps_of_rows_beside_each_other_are_refused(call, at):
    """Rows 8192 bytes apart, of 2000 bytes of logits and 2048 bytes of out."""
    refused(call, rlk.RLK_ERR_BAD_SHAPE, d=desc(ld_logits=4096), x=LOGITS,
            out=FakeTensor(PTR + at), ld=4096)


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


@pytest.mark.gpu
def test_rows_beside_each_other():
    n, v, pad = 9, 3001, 3016
    dev = torch.device("cuda")
    c = C.make_case(n, v, pad, 21, dev)
    rules = rlk.LogitRules(**c.rules)
    kw = dict(real_vocab=v, padded_vocab=pad)
    want = {t: rlk.process_logits(c.x, rules, out_dtype=t, **kw)
            for t in (torch.bfloat16, torch.float32)}
    lse = rlk.processed_forward(c.x, c.tgt, rules, c.mask, **kw)[1]
    grad = rlk.processed_backward(c.x, c.tgt, rules, c.mask, lse, c.g, c.gl,
                                  out_dtype=torch.bfloat16, **kw)
    for first in (0, 3 * pad):  # the logits in front of what is written, and behind
        wide = torch.zeros(n, 4 * pad, dtype=torch.bfloat16, device=dev)
        x = wide[:, first:first + pad]
        x.copy_(c.x)
        at = 0 if first else pad
        for dtype, out in ((torch.bfloat16, wide[:, at:at + pad]),
                           (torch.float32, wide.view(torch.float32)[:, at // 2:at // 2 + pad])):
            assert rlk.process_logits(x, rules, out_dtype=dtype, out=out, **kw) is out
            assert torch.equal(bits(out), bits(want[dtype]))
            assert torch.equal(bits(x), bits(c.x))
        rlk.rlk_logp_processed_bwd(rlk.make_desc(n, v, pad, 4 * pad, 1), x, rules.struct, c.tgt,
                                   c.mask.view(torch.uint8), lse, c.g, c.gl, wide[:, at:], 4 * pad,
                                   BF16, torch.empty(256, dtype=torch.uint8, device=dev))
        assert torch.equal(bits(wide[:, at:at + pad]), bits(grad))
    with pytest.raises(rlk.RlkError, match="overlaps the logits"):
        rlk.process_logits(wide[:, :pad], rules, out=wide[:, 8:8 + pad], **kw)
