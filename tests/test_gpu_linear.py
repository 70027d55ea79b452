"""Dense products with bias, activation and residual, and their gradients, against a plain form in
64 bits (tests/linear_cases.py).  Needs an MI355X."""
from __future__ import annotations

import math

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import linear_cases as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16 = torch.bfloat16


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


# tokens, in, out: few tokens in each width, tiles of either size, odd numbers of everything
SIZES = [(1, 64, 1), (1, 64, 8), (2, 128, 77), (3, 64, 4097), (16, 576, 130), (17, 320, 255),
         (32, 1088, 300), (33, 192, 64), (64, 448, 1001), (65, 64, 3), (100, 64, 129),
         (129, 192, 256), (300, 320, 515), (257, 1088, 64)]


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("m, k, n", SIZES)
def test_forward(m, k, n, act):
    print(f"case {m} {k} {n} {act}", flush=True)
    for bias, residual in ((torch.float32, True), (BF16, False), (None, True), (None, False)):
        c = C.make_case(m, k, n, act, m + k + n, DEV, bias, residual)
        y, saved = rlk.linear_forward(c.x, c.w, c.bias, c.residual, activation=act, cap=c.cap)
        assert saved is None and y.shape == (m, n)
        w = C.worst(y, *C.forward64(c))
        print(f"bias {bias} residual {residual}: error over bound {w:.3f}", flush=True)
        assert w <= 1.0
        y2, saved = rlk.linear_forward(c.x, c.w, c.bias, c.residual, activation=act, cap=c.cap,
                                       save=True)
        assert torch.equal(bits(y), bits(y2)) and (saved is None) == (act == "none")


@pytest.mark.parametrize("act", C.ACTS)
@pytest.mark.parametrize("m, k, n", SIZES)
def test_backward(m, k, n, act):
    for bias in (torch.float32, BF16):
        backward_case(m, k, n, act, bias)


def backward_case(m, k, n, act, bias):
    print(f"case {m} {k} {n} {act} bias {bias}", flush=True)
    c = C.make_case(m, k, n, act, 3 * m + k + n, DEV, bias, False)
    _, saved = rlk.linear_forward(c.x, c.w, c.bias, activation=act, cap=c.cap, save=True)
    kw = dict(activation=act, cap=c.cap)
    dx, dw, db = rlk.linear_backward(c.x, c.w, c.dy, saved, want_bias=True, **kw)
    rx, rw, rb = C.backward64(c)
    worst = [C.worst(dx, *rx), C.worst(dw, *rw), C.worst(db, *rb)]
    print("error over bound: dx {:.3f}, dW {:.3f}, db {:.3f}".format(*worst), flush=True)
    assert max(worst) <= 1.0
    # the same bits again, and when only one is asked for
    for want, full in (("x", dx), ("weight", dw), ("bias", db)):
        flags = {"want_" + name: name == want for name in ("x", "weight", "bias")}
        got = rlk.linear_backward(c.x, c.w, c.dy, saved, **flags, **kw)
        one = [t for t in got if t is not None]
        assert len(one) == 1 and torch.equal(bits(one[0]), bits(full)), want
    db16 = rlk.linear_backward(c.x, c.w, c.dy, saved, want_x=False, want_weight=False,
                               want_bias=True, bias_dtype=BF16, **kw)[2]
    assert torch.equal(bits(db16), bits(db.bfloat16()))


def whole(shape, lo, hi, gen, dtype=BF16):
    return torch.randint(lo, hi + 1, shape, generator=gen, device=DEV).to(dtype)


@pytest.mark.parametrize("m, k, n", SIZES + [(520, 64, 12300), (4100, 128, 900),
                                             (1030, 192, 13000)])
def test_whole_numbers_are_exact(m, k, n):
    """Small whole numbers: every sum is exact in fp32, so every output is the rounded exact one,
    and a term too many or too few shows."""
    print(f"case {m} {k} {n}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(m + n)
    x, w = whole((m, k), -2, 2, gen), whole((n, k), -2, 2, gen)
    b, r = whole((n,), -9, 9, gen, torch.float32), whole((m, n), -9, 9, gen)
    dy = whole((m, n), -3, 3, gen)
    y, _ = rlk.linear_forward(x, w, b, r)
    want = x.double() @ w.double().T + b.double() + r.double()
    assert torch.equal(y, want.bfloat16())
    dx, dw, db = rlk.linear_backward(x, w, dy, want_bias=True)
    assert torch.equal(dx, (dy.double() @ w.double()).bfloat16())
    assert torch.equal(dw, (dy.double().T @ x.double()).bfloat16())
    assert torch.equal(db, dy.double().sum(0).float())
    y, saved = rlk.linear_forward(x, w, b, r, activation="relu", save=True)
    z = x.double() @ w.double().T + b.double()
    assert torch.equal(y, (z.clamp_min(0) + r.double()).bfloat16())
    dz = dy.double() * (z > 0)
    dx, dw, db = rlk.linear_backward(x, w, dy, saved, activation="relu", want_bias=True)
    assert torch.equal(dx, (dz @ w.double()).bfloat16())
    assert torch.equal(dw, (dz.T @ x.double()).bfloat16())
    assert torch.equal(db, dz.sum(0).float())


def test_lmhead_logits():
    for m, k, v, pad in ((1, 64, 5, 5), (7, 128, 1000, 1024), (16, 64, 3001, 3003),
                         (90, 192, 1023, 1300), (300, 64, 999, 999), (65, 64, 100, 700)):
        for cap in (None, 5.0):
            c = C.make_case(m, k, pad, "none" if cap is None else "softcap", m + v, DEV,
                            torch.float32, False)
            c.w[v:] = math.nan  # padding rows are not read
            out = rlk.lmhead_logits(c.x, c.w, c.bias, cap=cap, real_vocab=v, padded_vocab=pad)
            assert out.shape == (m, pad) and (out[:, v:] == -math.inf).all()
            c.w, c.bias = c.w[:v], c.bias[:v]
            assert C.worst(out[:, :v], *C.forward64(c)) <= 1.0
            rows = pad if pad % 8 == 0 else (pad + 7) // 8 * 8
            assert out.stride(0) == rows or m == 1


def test_strides_and_what_lies_behind():
    """Residuals and gradients with rows of any stride; columns behind padded_out stay."""
    for m in (5, 200):
        c = C.make_case(m, 128, 77, "silu", m, DEV)
        want, saved = rlk.linear_forward(c.x, c.w, c.bias, c.residual, activation="silu",
                                         save=True)
        grads = rlk.linear_backward(c.x, c.w, c.dy, saved, activation="silu", want_bias=True)
        for width, at in ((80, 0), (88, 8), (96, 1), (79, 2)):
            wide = torch.full((m, width), math.nan, dtype=BF16, device=DEV)
            wide[:, at:at + 77] = c.residual
            got, _ = rlk.linear_forward(c.x, c.w, c.bias, wide[:, at:at + 77], activation="silu")
            assert torch.equal(bits(got), bits(want)), width
            wide[:, at:at + 77] = c.dy
            got = rlk.linear_backward(c.x, c.w, wide[:, at:at + 77], saved, activation="silu",
                                      want_bias=True)
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, grads)), width
        out = torch.full((m, 104), 7.0, dtype=BF16, device=DEV)
        d = rlk.rlk_linear_desc(m, 128, 77, 79, 104, 0, 80, 0, 0, 0, 0.0)
        rlk.rlk_linear_fwd(d, c.x, c.w, c.bias, None, out, None)
        assert (out[:, 77:79] == -math.inf).all() and (out[:, 79:] == 7.0).all()


def test_extreme_values():
    """Far positive and negative z reach each activation's ends, and NaN stays NaN."""
    for act, low, high in (("relu", 0, 2.0 ** 20), ("gelu", 0, 2.0 ** 20),
                           ("gelu_tanh", 0, 2.0 ** 20), ("silu", 0, 2.0 ** 20),
                           ("softcap", -5.0, 5.0)):
        for m in (1, 70):
            x = torch.zeros(m, 64, dtype=BF16, device=DEV)
            x[:, 0], x[:, 1] = 1024.0, math.nan
            w = torch.zeros(24, 64, dtype=BF16, device=DEV)
            w[:8, 0], w[8:16, 0] = 1024.0, -1024.0
            x[:, 1] = 0.0
            cap = 5.0 if act == "softcap" else None
            y, saved = rlk.linear_forward(x, w, activation=act, cap=cap, save=True)
            assert (y[:, :8] == high).all() and (y[:, 8:16] == low).all() and (y[:, 16:] == 0).all()
            dy = torch.ones_like(y)
            dx, dw, db = rlk.linear_backward(x, w, dy, saved, activation=act, cap=cap,
                                             want_bias=True)
            assert (db[:8] == (0 if act == "softcap" else m)).all() and (db[8:16] == 0).all()
            assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
            x[0, 0] = math.nan
            y, _ = rlk.linear_forward(x, w, activation=act, cap=cap)
            assert y[0].isnan().all() and not y[1:].isnan().any()


def test_autograd():
    for m, n in ((3, 77), (150, 200)):
        for act in C.ACTS:
            for bias, residual in ((BF16, True), (torch.float32, False), (None, True)):
                c = C.make_case(m, 192, n, act, 7, DEV, bias, residual)
                leaves = [t.requires_grad_(True) for t in (c.x, c.w, c.bias, c.residual)
                          if t is not None]
                y = rlk.head_linear(c.x, c.w, c.bias, c.residual, activation=act, cap=c.cap)
                got = torch.autograd.grad(y, leaves, c.dy)
                with torch.no_grad():
                    want_y, saved = rlk.linear_forward(c.x, c.w, c.bias, c.residual,
                                                       activation=act, cap=c.cap, save=True)
                    want = rlk.linear_backward(c.x, c.w, c.dy, saved, activation=act, cap=c.cap,
                                               want_bias=bias is not None,
                                               bias_dtype=bias or torch.float32)
                assert torch.equal(bits(y.detach()), bits(want_y))
                want = [t for t in want if t is not None] + ([c.dy] if residual else [])
                assert len(got) == len(want)
                assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
                assert [t.dtype for t in got] == [t.dtype for t in leaves]
    # an expanded gradient, a frozen weight, and no second derivatives
    c = C.make_case(5, 64, 24, "silu", 8, DEV, None, False)
    x = c.x.requires_grad_(True)
    y = rlk.head_linear(x, c.w, activation="silu")
    dx, = torch.autograd.grad(y.sum(), x, retain_graph=True)
    _, saved = rlk.linear_forward(c.x.detach(), c.w, activation="silu", save=True)
    want = rlk.linear_backward(c.x.detach(), c.w, torch.ones_like(c.dy), saved, activation="silu",
                               want_weight=False)[0]
    assert torch.equal(bits(dx), bits(want))
    with pytest.raises(RuntimeError):
        first, = torch.autograd.grad(y.sum(), x, create_graph=True)
        torch.autograd.grad(first.float().sum(), x)


def test_no_tokens():
    x = torch.zeros(0, 64, dtype=BF16, device=DEV)
    w = torch.ones(9, 64, dtype=BF16, device=DEV)
    y, saved = rlk.linear_forward(x, w, torch.ones(9, device=DEV), activation="silu", save=True)
    assert y.shape == (0, 9)
    dx, dw, db = rlk.linear_backward(x, w, y, saved, activation="silu", want_bias=True)
    assert dx.shape == (0, 64) and (bits(dw) == 0).all() and (bits(db) == 0).all()
    assert rlk.lmhead_logits(x, w, real_vocab=9).shape == (0, 9)


@pytest.mark.parametrize("m", [1, 70])
def test_the_smallest_and_the_largest_cap(m):
    """x picks one column of the weight, so z is exact.  At 1e30 z / cap stays normal and the soft
    cap is z but for four roundings (1 / cap, z / cap, tanh's quotient, the product) of 2^-23 at
    most, its slope 4 (1/2)^2 but for three; at 1e-30 they are +-cap but for four and 0."""
    torch.manual_seed(4)
    w = (torch.rand(96, 64, device=DEV) + 0.5) * torch.randn(96, 64, device=DEV).sign()
    w = w.bfloat16()
    x = torch.zeros(m, 64, dtype=torch.bfloat16, device=DEV)
    x[:, 5] = 1.0
    z = w[:, 5].double().expand(m, -1)
    dy = torch.randn(m, 96, device=DEV).bfloat16()
    for cap, want, slope in ((1e30, z, 1.0), (1e-30, z.sign() * 1e-30, 0.0)):
        y, saved = rlk.linear_forward(x, w, torch.zeros(96, device=DEV), activation="softcap",
                                      cap=cap, save=True)
        assert ((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -20)).all()
        _, _, db = rlk.linear_backward(x, w, dy, saved, activation="softcap", cap=cap,
                                       want_bias=True)
        exact = dy.double().sum(0) * slope
        # (the sum of m terms: m roundings of 2^-24)
        bound = dy.double().abs().sum(0) * slope * (2.0 ** -20 + m * 2.0 ** -24)
        assert ((db.double() - exact).abs() <= bound).all()


@pytest.mark.parametrize("m", [1000, 850])
def test_a_last_round_in_half_tiles(m):
    """1320 of the largest tiles are five rounds of the chip and 40 more, of which the half behind
    the last token (850: from 896 on) has nothing to do."""
    n, k = 84480, 64
    c = C.make_case(m, k, n, "silu", 9 + m, DEV, BF16, True)
    y, saved = rlk.linear_forward(c.x, c.w, c.bias, c.residual, activation="silu", save=True)
    for at in range(0, n, 16896):  # the bounds by pieces
        here = slice(at, at + 16896)
        piece = C.Case(c.x, c.w[here], c.bias[here], c.residual[:, here], c.dy[:, here], "silu")
        assert C.worst(y[:, here], *C.forward64(piece)) <= 1.0
        z, ez = C.product64(piece)
        # (fp16's half step)
        assert ((saved[:, here].double() - z).abs() <= ez + 2.0 ** -11 * (z.abs() + ez)
                + 2.0 ** -25).all()
    # the same bits as of the last outputs alone, which take other tiles
    last, _ = rlk.linear_forward(c.x, c.w[-4096:].contiguous(), c.bias[-4096:].contiguous(),
                                 c.residual[:, -4096:], activation="silu")
    assert torch.equal(bits(y[:, -4096:]), bits(last))
