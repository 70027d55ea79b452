"""The bytes of the 8-bit cast, signs of zeros among them.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import fp8_cases as F

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("block_rows", [1, 128])
def test_bytes(block_rows):
    """Blocks from the smallest scale to the largest: a zero keeps its sign, whichever way its
    block's quotients are taken, and so does what rounds to zero."""
    rows = []
    for e in (-133, -126, -100, -70, -50, -20, 0, 20, 100, 127):
        r = torch.randn(256, generator=torch.Generator().manual_seed(e + 200)) * 2.0 ** (e - 2)
        r[3] = 2.0 ** e
        r[::5] = 0.0
        r[::10] = -0.0
        r[1::10] *= 2.0 ** -12  # rounds to a zero of its sign
        rows.append(r)
    x = torch.stack(rows)
    if block_rows == 128:
        x = x.repeat_interleave(128, 0)
    x = x.to(torch.bfloat16).to(DEV)
    assert (x.view(torch.int16) == -32768).any() and x.float().isfinite().all()
    q, scale = rlk.quantize_fp8(x, block_rows)
    qr, sr = F.cast64(x, block_rows)
    assert torch.equal(scale.double(), sr)
    want = qr.float().to(torch.float8_e4m3fn)
    assert torch.equal(want.double(), qr)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))
