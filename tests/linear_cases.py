"""Seeded dense products with their epilogue, their plain form and gradients in 64 bits, and
the error a kernel with bf16 operands and fp32 sums may make (arithmetic only)."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

HALF_BF16 = 2.0 ** -8   # half a step, relative
HALF_FP16 = 2.0 ** -11
H = 2.0 ** -24          # of fp32
CAP = 5.0
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "softcap")


@dataclass
class Case:
    x: torch.Tensor
    w: torch.Tensor
    bias: torch.Tensor | None
    residual: torch.Tensor | None
    dy: torch.Tensor
    act: str

    @property
    def cap(self):
        return CAP if self.act == "softcap" else None


def make_case(m, k, n, act, seed, device, bias=torch.float32, residual=True):
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=device)

    return Case(normal(m, k).bfloat16(), (normal(n, k) * (2.0 / k ** 0.5)).bfloat16(),
                None if bias is None else normal(n).to(bias),
                normal(m, n).bfloat16() if residual else None, normal(m, n).bfloat16(), act)


def act64(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), which does not cancel for u far below 0
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "softcap":
        return CAP * torch.tanh(z / CAP)
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) \
            + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        u = c * (z + 0.044715 * z ** 3)
        return torch.sigmoid(u) * (1.0 + z * torch.sigmoid(-u) * c * (1.0 + 3 * 0.044715 * z * z))
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if act == "softcap":
        return 1.0 / torch.cosh(z / CAP) ** 2
    return torch.ones_like(z)


def product64(c: Case):
    """z and the bound on its error: K products and the bias, summed in fp32."""
    x, w = c.x.double(), c.w.double()
    z = x @ w.T
    err = (x.shape[1] + 2) * H * (x.abs() @ w.abs().T)
    if c.bias is not None:
        z = z + c.bias.double()
        err = err + H * z.abs()
    return z, err


def moved(f, z, d):
    """How far f moves when z moves by up to d (f is monotonous over so short a way, or nearly:
    a tenth more)."""
    at = f(z)
    return 1.1 * torch.maximum((f(z + d) - at).abs(), (f(z - d) - at).abs())


def of_exponentials(z):
    """Relative error of an activation's own arithmetic: the argument of its exponential is
    rounded a few times (which counts times its size: z^2 at most, or the cubic polynomial's
    size), the rest takes 16 half steps; a tanh's difference next to 0 costs up to 128."""
    return H * (144 + 4 * z * z + 16 * (z + 0.044715 * z ** 3).abs())


def forward64(c: Case):
    z, ez = product64(c)
    y = act64(z, c.act)
    err = moved(lambda t: act64(t, c.act), z, ez)
    if c.act not in ("none", "relu"):
        err = err + y.abs() * of_exponentials(z) + 1e-37
    if c.residual is not None:
        y = y + c.residual.double()
        err = err + H * y.abs()
    return y, err + HALF_BF16 * (y.abs() + err)


def backward64(c: Case):
    """((dx, its bound), (dW, its bound), (db, its bound)), db's for an fp32 bias."""
    z, ez = product64(c)
    x, w, dy = c.x.double(), c.w.double(), c.dy.double()
    s = slope64(z, c.act)
    dz = dy * s
    es = torch.zeros_like(z)
    if c.act != "none":
        # z is kept in fp16: half a step, or of its smallest ones; in fp32 with such a bias
        exact = c.bias is not None and c.bias.dtype == torch.float32
        kept = H * z.abs() if exact else \
            HALF_FP16 * z.abs() + 2.0 ** -25 * (CAP if c.act == "softcap" else 1.0)
        es = moved(lambda t: slope64(t, c.act), z, kept + ez)
        if c.act != "relu":
            es = es + of_exponentials(z) * (s.abs() + 0.25)
    e_sum = dy.abs() * es + H * dz.abs()
    e_dz = e_sum + HALF_BF16 * (dz.abs() + e_sum) if c.act != "none" else torch.zeros_like(z)
    m, n = z.shape
    dx, dw, db = dz @ w, dz.T @ x, dz.sum(0)
    e_dx = e_dz @ w.abs() + (n + 2) * H * (dz.abs() @ w.abs())
    e_dw = e_dz.T @ x.abs() + (m + 2) * H * (dz.abs().T @ x.abs())
    e_db = e_sum.sum(0) + (m + 2) * H * dz.abs().sum(0)
    return ((dx, e_dx + HALF_BF16 * (dx.abs() + e_dx)), (dw, e_dw + HALF_BF16 * (dw.abs() + e_dw)),
            (db, e_db))


def worst(got, want, err):
    d = (got.double() - want).abs()
    assert torch.isfinite(d).all(), "non-finite values"
    assert (d[err == 0] == 0).all(), "an element that must be exact is not"
    return float((d / err.clamp_min(1e-300)).max()) if d.numel() else 0.0
