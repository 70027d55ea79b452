"""The logit rules' statistics and gradient where logits lie far out: pieces of a row held down by a
large finite number, as masks that add one do, rows whose logits are large altogether, and
temperatures next to 0.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import process_cases as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
FAR = (1e6, 1.6e7, 1.7e7, 1e8, 1.5e9, 3e9, 1e10, 1e12, 1e20, 1e28, 9e29, 1.1e30, 1e37)


def forward(c):
    return rlk.processed_forward(c.x, c.tgt, rlk.LogitRules(**c.rules), c.mask, real_vocab=c.v,
                                 padded_vocab=c.pad)


def backward(c, lse):
    return rlk.processed_backward(c.x, c.tgt, rlk.LogitRules(**c.rules), c.mask, lse, c.g, c.gl,
                                  real_vocab=c.v, padded_vocab=c.pad)


def checked(c):
    logp, lse = forward(c)
    want_logp, want_lse, _, _, e_logp, e_lse, _ = C.logp64(c)
    assert C.worst(logp, want_logp, e_logp) <= 1.0 and C.worst(lse, want_lse, e_lse) <= 1.0
    return lse


@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("by_bias", [False, True])
def test_pieces_held_down(far, by_bias):
    """Columns 2048 to 6143, two whole pieces, and some single ones lie at -far: the row's
    statistics and gradient are those of the other columns."""
    print(f"case {far} by bias {by_bias}", flush=True)
    n, v = 6, 9001
    c = C.make_case(n, v, 9008, 31, DEV, "none")
    c.tgt[:] = torch.tensor([0, 5, 2047, 6144, 9000, 7000])
    down = torch.zeros(v, dtype=torch.bool, device=DEV)
    down[2048:6144] = True
    down[7001:7010] = True
    if by_bias:
        c.rules = {"bias": torch.where(down, -far, 0.0)}
    else:
        c.x[:, :v] = torch.where(down, -far, c.x[:, :v].float()).bfloat16()
    lse = checked(c)
    want, err = C.gradient64(c, c.g, c.gl, C.H)
    d = backward(c, lse)
    assert C.worst(d, want, err) <= 1.0
    assert (d[:, :v][:, down] == 0).all()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("far", FAR)
def test_rows_far_out(far, sign):
    """Every logit is large and one lies an eighth above the others: it has all of the weight."""
    print(f"case {far} {sign}", flush=True)
    n, v = 4, 5000
    c = C.make_case(n, v, v, 32, DEV, "none")
    top = torch.tensor([0, 2500, 4999, 100], device=DEV)
    c.x[:] = sign * far * (1.0 if sign > 0 else 1.125)
    rows = torch.arange(n, device=DEV)
    c.x[rows, top] = sign * far * (1.125 if sign > 0 else 1.0)
    c.tgt[:] = top.int()
    c.tgt[3] = 7
    c.mask[:] = True
    lse = checked(c)
    assert torch.equal(lse, c.x[rows, top].float())
    d = backward(c, lse)
    # p = 1 of the top as exp2(r) (gl - g) exp2(-r), r what rounding took from LSE log2 e: two
    # exponentials of 2 half steps each, gl - g and two products of one; then the sum with g
    coef, g = c.gl.double() - c.g.double(), torch.where(rows == 3, 0.0, c.g.double())
    want = torch.zeros(n, v, dtype=torch.float64, device=DEV)
    want[rows, top] = coef + g
    want[3, 7] = c.g[3].double()
    bound = torch.zeros_like(want)
    bound[rows, top] = 1.001 * (7 * C.H * coef.abs() + torch.where(rows == 3, 0.0,
                                                                   C.H * (coef + g).abs()))
    assert C.worst(d, want, bound) <= 1.0


@pytest.mark.parametrize("temperature", [1e-4, 1e-6, 1e-8, 1e-10, 1e-20, 1e-30])
def test_temperatures_next_to_0(temperature):
    print(f"case {temperature}", flush=True)
    n, v = 5, 6000
    c = C.make_case(n, v, v, 33, DEV, "none")
    top = c.x.float().amax(1, keepdim=True)
    c.x[:] = torch.where(c.x.float() > top - 0.5, 1.0, c.x.float()).bfloat16()
    at = torch.tensor([3, 2048, 4095, 4096, 5999], device=DEV)
    rows = torch.arange(n, device=DEV)
    c.x[rows, at] = 16.0
    c.tgt[:], c.mask[:] = at.int(), True
    c.rules = {"temperature": torch.full((n,), temperature, device=DEV)}
    lse = checked(c)
    logp, _ = forward(c)
    assert (logp == 0).all()
    d = backward(c, lse)
    others = torch.ones(n, v, dtype=torch.bool, device=DEV)
    others[rows, at] = False
    assert (d[others] == 0).all() and torch.isfinite(d).all()
