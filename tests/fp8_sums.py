"""How far an 8-bit product may be from 64 bits when its sums are held in fp32, root mean
square over many outputs, for the LM-head's 8-bit tests (arithmetic only)."""
from __future__ import annotations

import torch

from tests import fp8_cases as F

HALF_F32 = 2.0 ** -24


def operands(n, k, v, seed, device):
    """Hidden states and a weight as a model has them, in 8 bits: ((q, scale), (q, scale))."""
    gen = torch.Generator(device=device).manual_seed(seed)
    h = torch.randn((n, k), generator=gen, device=device)
    w = torch.randn((v, k), generator=gen, device=device) * (1.3 / k ** 0.5)
    out = []
    for x, rows in ((h, 1), (w, F.BLOCK)):
        q, s = F.cast64(x.to(torch.bfloat16), rows)
        out.append((q.float().to(torch.float8_e4m3fn), s.float()))
    return out


def blocks64(hq, hs, wq, ws):
    """h . w^T of each block of 128 columns in 64 bits, and the sums of its magnitudes:
    two [blocks, n, v] tensors."""
    h, w = F.value64(hq, hs, 1), F.value64(wq, ws, F.BLOCK)
    h = h.unflatten(1, (-1, F.BLOCK)).transpose(0, 1).contiguous()
    w = w.unflatten(1, (-1, F.BLOCK)).permute(1, 2, 0).contiguous()
    return torch.bmm(h, w), torch.bmm(h.abs(), w.abs())


def product64(hq, hs, wq, ws):
    """(z, tolerance): z in 64 bits [n, v] and the root mean square over all its elements that
    an error of fp32 sums does not exceed.

    A product of two e4m3 values has 8 bits and is exact.  A block's 128 products are added in
    fp32 in some order: each addition is off by half a step (2^-24) of a partial sum, which
    the sum of the block's magnitudes bounds.  The block's sum is multiplied by the product of
    its two scales (rounded: half a step of the scaled sum) and added to the others (half a
    step of the running sum).  These roundings have no sign of their own, so their squares
    add up."""
    z, size = blocks64(hq, hs, wq, ws)
    running = z.cumsum(0)
    square = (F.BLOCK * size ** 2 + z ** 2 + running ** 2).sum(0) * HALF_F32 ** 2
    return running[-1], float(square.mean().sqrt())


def rms(x):
    return float(x.double().square().mean().sqrt())
