"""Seeded LM-head cases and the plain form of its gradients in 64 bits, with the error a
bf16 kernel may make, for the LM-head tests (input synthesis and arithmetic only)."""
from __future__ import annotations

from dataclasses import dataclass

import torch

IGNORE = -100
HALF_BF16 = 2.0 ** -8   # half a step of bf16, relative
HALF_F32 = 2.0 ** -24


@dataclass
class Case:
    h: torch.Tensor     # bf16 [N, K]
    w: torch.Tensor     # bf16 [rows, K]; rows >= v_real hold random bit patterns
    tgt: torch.Tensor   # int32 [N]
    mask: torch.Tensor  # bool [N]
    g: torch.Tensor     # fp32 [N]
    gl: torch.Tensor    # fp32 [N]
    v_real: int

    @property
    def active(self):
        return self.mask & (self.tgt != IGNORE)


def garbage(shape, gen, device):
    return torch.randint(-32768, 32768, shape, generator=gen, device=device,
                         dtype=torch.int32).to(torch.int16).view(torch.bfloat16)


def make_case(n, k, v_real, v_pad, seed, device, mask_keep=0.8, ignore_frac=0.1, peaked=0.5,
              scale=1.0):
    """Half the tokens are likely under the model (their logit stands about 8 above)."""
    gen = torch.Generator(device=device).manual_seed(seed)
    sigma = 1.3 / k ** 0.5
    w = (torch.randn((v_pad, k), generator=gen, device=device) * sigma).to(torch.bfloat16)
    tgt = torch.randint(0, v_real, (n,), generator=gen, device=device, dtype=torch.int32)
    h = torch.randn((n, k), generator=gen, device=device)
    lean = (torch.rand(n, generator=gen, device=device) < peaked).float() * 8.0 / (k * sigma ** 2)
    h = (h + lean[:, None] * w[tgt.long()].float()).to(torch.bfloat16)
    if v_pad > v_real:
        w[v_real:] = garbage((v_pad - v_real, k), gen, device)
    mask = torch.rand(n, generator=gen, device=device) < mask_keep
    tgt[torch.rand(n, generator=gen, device=device) < ignore_frac] = IGNORE
    g = torch.randn(n, generator=gen, device=device) * scale
    gl = torch.randn(n, generator=gen, device=device) * (0.3 * scale)
    return Case(h, w, tgt, mask, g, gl, v_real)


def forward64(c: Case):
    """(logp, LSE, z) in 64 bits; logp is 0 on rows that are not active."""
    z = c.h.double() @ c.w[:c.v_real].double().T
    lse = torch.logsumexp(z, 1)
    at = torch.where(c.active, c.tgt, 0).long()[:, None]
    logp = torch.where(c.active, z.gather(1, at)[:, 0] - lse, 0.0)
    return logp, lse, z


def gradients64(c: Case, g, gl):
    """(dh, dW) in 64 bits and, for each, the bound on a kernel's error:

    * z is a sum of K products in fp32: off by at most (K + 2) half steps of the sum of
      their magnitudes, and so is LSE by no more than the largest of its z's error plus a
      few steps of its own; p = exp(z - LSE) is off by those relative errors, by the
      rounding of z - LSE and of its product with log2 e (4 half steps of |z - LSE|), and
      by 8 half steps of the exponential and the products that follow;
    * dz is rounded to bf16 once (half a step), the products are summed in fp32 over the
      vocabulary (or the tokens), one half step of the magnitudes' sum per term;
    * the result is rounded to bf16 once.
    """
    logp, lse, z = forward64(c)
    h, w = c.h.double(), c.w[:c.v_real].double()
    a = c.active
    g = torch.where(a, g.double(), 0.0) if g is not None else torch.zeros_like(lse)
    gl = gl.double() if gl is not None else torch.zeros_like(lse)
    reached = (g != 0) | (gl != 0)
    k, n, v = h.shape[1], h.shape[0], c.v_real
    p = (z - lse[:, None]).exp()
    dz = (gl - g)[:, None] * p
    rows = torch.arange(n, device=z.device)
    at = torch.where(a, c.tgt, 0).long()
    dz[rows, at] += g
    z_err = (k + 2) * HALF_F32 * (h.abs() @ w.abs().T)
    rel = (z_err + z_err.amax(1, keepdim=True) + 8 * HALF_F32 * lse.abs()[:, None]
           + 4 * HALF_F32 * (z - lse[:, None]).abs() + 8 * HALF_F32)
    dz_err = HALF_BF16 * dz.abs() + rel * p * (gl.abs() + g.abs())[:, None]
    dz = torch.where(reached[:, None], dz, 0.0)
    dz_err = torch.where(reached[:, None], dz_err, 0.0)
    h = torch.where(reached[:, None], h, 0.0)  # rows that no term reaches hold anything
    dh, dw = dz @ w, dz.T @ h
    dh_err = dz_err @ w.abs() + (v + 2) * HALF_F32 * (dz.abs() @ w.abs()) + HALF_BF16 * dh.abs()
    dw_err = dz_err.T @ h.abs() + (n + 2) * HALF_F32 * (dz.abs().T @ h.abs()) \
        + HALF_BF16 * dw.abs()
    full = torch.zeros((c.w.shape[0], k), dtype=torch.float64, device=z.device)
    full_err = full.clone()
    full[:v], full_err[:v] = dw, dw_err
    return dh, dh_err, full, full_err


def worst(got, want, err):
    """The largest error over its bound (an element with a zero bound has to be equal)."""
    d = (got.double() - want).abs()
    assert torch.isfinite(d).all(), "non-finite values"
    assert (d[err == 0] == 0).all(), "an element that must be exact is not"
    return float((d / err.clamp_min(1e-300)).max()) if d.numel() else 0.0
