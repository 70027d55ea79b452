"""The bound of tests/fp8_sums.py tells fp32 sums from products that keep fewer bits: sums in
fp32 stay within it, planted losses do not (arithmetic on the CPU)."""
from __future__ import annotations

import pytest
import torch

from tests import fp8_cases as F
from tests import fp8_sums as S

KS = [1024, 4096]


def cut_in_groups(hq, hs, wq, ws, group=8, keep=13):
    """z with each product cut towards zero `keep` bits below the largest exponent among the
    products of its `group` columns."""
    f = F.value64(hq, hs, 1), F.value64(wq, ws, F.BLOCK)
    z = torch.zeros((hq.shape[0], wq.shape[0]), dtype=torch.float64)
    for b in range(hq.shape[1] // F.BLOCK):
        at = slice(b * F.BLOCK, (b + 1) * F.BLOCK)
        p = hq[:, None, at].double() * wq[None, :, at].double()
        g = p.unflatten(2, (-1, group))
        e = torch.floor(torch.log2(hq[:, at].double().abs().clamp_min(2.0 ** -6)))[:, None] \
            + torch.floor(torch.log2(wq[:, at].double().abs().clamp_min(2.0 ** -6)))[None]
        e = torch.where(p == 0, -torch.inf, e).unflatten(2, (-1, group))
        unit = torch.exp2(e.amax(3, keepdim=True).clamp_min(-64) - keep)
        total = (torch.trunc(g / unit) * unit).sum((2, 3))
        z += total * (hs[:, b, None].double() * ws[0, b].double())
    assert f[0].shape[1] == f[1].shape[1]
    return z


@pytest.mark.parametrize("k", KS)
def test_bound_tells_sums_in_fp32_from_less(k):
    (hq, hs), (wq, ws) = S.operands(48, k, 64, k, "cpu")
    z, tol = S.product64(hq, hs, wq, ws)
    # a block's sum in fp32, in ascending columns, scaled and added as fp32
    acc = torch.zeros(z.shape)
    for b in range(k // F.BLOCK):
        s = torch.zeros(z.shape)
        for c in range(b * F.BLOCK, (b + 1) * F.BLOCK):
            s += hq[:, c, None].float() * wq[None, :, c].float()
        acc += s * (hs[:, b, None] * ws[0, b])
    assert S.rms(acc - z) <= tol
    # scales that lost bits, and products cut beside larger ones
    low = hs.to(torch.bfloat16).float()
    assert S.rms(S.product64(hq, low, wq, ws)[0] - z) > 10 * tol
    assert S.rms(cut_in_groups(hq, hs, wq, ws) - z) > 1.5 * tol
