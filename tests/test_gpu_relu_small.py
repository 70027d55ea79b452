"""ReLU's slope is z's sign, however small z is and in however few bits it is kept.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16 = torch.bfloat16


@pytest.mark.parametrize("bias", [None, BF16, torch.float32])
@pytest.mark.parametrize("exponent", [-24, -25, -26, -40, -100])
# few tokens with few outputs and with many, and tiles
@pytest.mark.parametrize("m, n", [(1, 77), (40, 300), (20, 9000), (70, 130), (300, 1001)])
def test_small_z(m, n, exponent, bias):
    """x picks one column of a weight of whole multiples of one power of two, so z, every sum and
    every result are exact."""
    print(f"case {m} {n} 2^{exponent} bias {bias}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(m + n)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=gen, device=DEV).double()

    x = torch.zeros(m, 64, dtype=BF16, device=DEV)
    x[:, 5] = 1.0
    w = (whole(-1, 1, n, 64) * 2.0 ** exponent).to(BF16)
    dy = whole(-2, 2, m, n).to(BF16)
    b = None if bias is None else torch.zeros(n, dtype=bias, device=DEV)
    z = w[:, 5].double().expand(m, n)
    y, saved = rlk.linear_forward(x, w, b, activation="relu", save=True)
    assert saved.dtype == (torch.float32 if bias == torch.float32 else torch.float16)
    assert torch.equal(y.double(), z.clamp_min(0))
    assert torch.equal(saved[:, :n] > 0, z > 0)
    dz = dy.double() * (z > 0)
    dx, dw, db = rlk.linear_backward(x, w, dy, saved, activation="relu", want_bias=True)
    assert torch.equal(db.double(), dz.sum(0)) and (db != 0).any()
    assert torch.equal(dx, (dz @ w.double()).to(BF16))
    assert torch.equal(dw, (dz.T @ x.double()).to(BF16))
