"""The 8-bit cast and product in 64 bits, for the LM-head's 8-bit tests (arithmetic only)."""
from __future__ import annotations

import torch

BLOCK = 128
HALF_F32 = 2.0 ** -24


def e4m3(x):
    """x (float64) to the nearest e4m3 value, to even; 3 fraction bits, exponents from -6."""
    unit = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / unit) * unit


def cast64(x, block_rows):
    """(q, scale) of bf16 x as float64 tensors: quotients rounded once to fp32."""
    n, k = x.shape
    rows = -(-n // block_rows)
    pad = torch.zeros((rows * block_rows, k), dtype=torch.float64, device=x.device)
    pad[:n] = x.double()
    b = pad.view(rows, block_rows, k // BLOCK, BLOCK)
    top = b.abs().amax((1, 3))
    scale = (top / 448.0).float().double()
    scale = torch.where(scale < 2.0 ** -126, 2.0 ** -126, scale)  # NaN stays
    q = e4m3((b / scale[:, None, :, None]).float().double())
    return q.reshape(-1, k)[:n], scale


def value64(q, scale, block_rows):
    ids = torch.arange(q.shape[0], device=q.device) // block_rows
    return q.double() * scale.double()[ids].repeat_interleave(BLOCK, 1)


def group_error(hq, hs, wq, ws):
    """What the matrix cores may lose of each element of h . w^T as they line products up.

    They add 8-bit products in groups of 8 columns and cut each towards zero 13 bits below
    the largest exponent of its group (the sum of its factors' exponents, a subnormal
    counted as 2^-6, products of zero left out; test_products_meet_in_groups_of_eight pins
    this).  So of seven products less than 2^-13 of max |h'||w'| each is lost, where x' is x, or
    2^-6 if that is more; the largest loses nothing.  A group's sum and the sum over groups
    are fp32."""
    def floored(q, s, rows):
        a = q.double().abs()
        return value64(torch.where(a > 0, a.clamp_min(2.0 ** -6), a), s, rows)
    h, w = floored(hq, hs, 1), floored(wq, ws, BLOCK)
    lost = torch.zeros((h.shape[0], w.shape[0]), dtype=torch.float64, device=h.device)
    for k in range(0, h.shape[1], 8):
        top = h[:, k, None] * w[None, :, k]
        for i in range(k + 1, k + 8):
            top = torch.maximum(top, h[:, i, None] * w[None, :, i])
        lost += top
    return 7 * 2.0 ** -13 * lost


def product64(hq, hs, wq, ws, v_real):
    """z in 64 bits and the bound on its error: what the matrix cores lose (group_error); a
    block's sums in fp32 (16 groups, taken: 128 roundings), two scales multiplied and the
    result added up over K / 128 blocks, each at most half a step of the magnitudes' sum."""
    wq, ws = wq[:v_real], ws[:-(-v_real // BLOCK)]
    h, w = value64(hq, hs, 1), value64(wq, ws, BLOCK)
    k = h.shape[1]
    z = h @ w.T
    return z, group_error(hq, hs, wq, ws) + (BLOCK + k // BLOCK + 3) * HALF_F32 * (
        h.abs() @ w.abs().T)
