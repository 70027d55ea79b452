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


def product64(hq, hs, wq, ws, v_real):
    """z in 64 bits and the bound on its error in fp32: a block's 128 products summed (128
    roundings at most), two scales multiplied and the result added up over K / 128 blocks,
    each at most half a step of the magnitudes' sum."""
    h, w = value64(hq, hs, 1), value64(wq, ws, BLOCK)[:v_real]
    k = h.shape[1]
    z = h @ w.T
    return z, (BLOCK + k // BLOCK + 3) * HALF_F32 * (h.abs() @ w.abs().T)
