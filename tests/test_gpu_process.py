"""The logit rules, and the selected-token log-probability under them with its gradient, against a
plain form in 64 bits (tests/process_cases.py).  Needs an MI355X."""
from __future__ import annotations

import math

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import process_cases as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def rules(c):
    return rlk.LogitRules(**c.rules)


def forward(c, **kw):
    return rlk.processed_forward(c.x, c.tgt, rules(c), c.mask, real_vocab=c.v,
                                 padded_vocab=c.pad, **kw)


def backward(c, lse, g, gl, **kw):
    return rlk.processed_backward(c.x, c.tgt, rules(c), c.mask, lse, g, gl, real_vocab=c.v,
                                  padded_vocab=c.pad, **kw)


SIZES = [(1, 1, 1), (1, 7, 9), (3, 33, 40), (3, 2048, 2048), (2, 2049, 2056), (5, 8191, 8200),
         (4, 8193, 9000), (17, 20000, 20481), (2, 70001, 70001), (300, 1030, 1040)]


@pytest.mark.parametrize("kind", C.KINDS)
@pytest.mark.parametrize("n, v, pad", SIZES)
def test_processed_logits(n, v, pad, kind):
    print(f"case {n} {v} {pad} {kind}", flush=True)
    c = C.make_case(n, v, pad, 5 + n + v, DEV, kind)
    y, _, err = C.processed64(c)
    for dtype, half in ((torch.bfloat16, C.HALF_BF16), (torch.float32, C.H)):
        out = rlk.process_logits(c.x, rules(c), real_vocab=v, padded_vocab=pad, out_dtype=dtype)
        assert out.shape == (n, pad) and out.dtype == dtype
        bound = err + half * (torch.where(y == -math.inf, 0.0, y).abs() + err)
        bound = torch.where(y == -math.inf, 0.0, bound + C.TINY)
        w = C.worst(out[:, :v], y, bound)
        print(f"{dtype}: error over bound {w:.3f}", flush=True)
        assert w <= 1.0
        assert (out[:, v:] == -math.inf).all()
        again = rlk.process_logits(c.x, rules(c), real_vocab=v, padded_vocab=pad, out_dtype=dtype)
        assert torch.equal(bits(out), bits(again))


@pytest.mark.parametrize("kind", C.KINDS)
@pytest.mark.parametrize("n, v, pad", SIZES)
def test_processed_logp_and_gradient(n, v, pad, kind):
    print(f"case {n} {v} {pad} {kind}", flush=True)
    c = C.make_case(n, v, pad, 77 + n + v, DEV, kind)
    logp, lse = forward(c)
    want_logp, want_lse, _, _, e_logp, e_lse, _ = C.logp64(c)
    a, b = C.worst(logp, want_logp, e_logp), C.worst(lse, want_lse, e_lse)
    print(f"error over bound: logp {a:.3f}, lse {b:.3f}", flush=True)
    assert a <= 1.0 and b <= 1.0
    for g, gl in ((c.g, None), (None, c.gl), (c.g, c.gl)):
        for dtype, half in ((torch.bfloat16, C.HALF_BF16), (torch.float32, C.H)):
            d = backward(c, lse, g, gl, out_dtype=dtype)
            want, err = C.gradient64(c, g, gl, half)
            w = C.worst(d, want, err)
            print(f"gradient {dtype} g {g is not None} gl {gl is not None}: {w:.3f}", flush=True)
            assert w <= 1.0
            assert (bits(d[:, v:]) == 0).all()  # +0 in the padding
            assert torch.equal(bits(d), bits(backward(c, lse, g, gl, out_dtype=dtype)))


def test_long_histories_and_every_place_of_their_ends():
    """A row's history begins and ends at any place of a vector; long ones take several rounds."""
    n, v = 12, 9000
    c = C.make_case(n, v, v, 3, DEV, "all", longest=9000)
    begin = torch.tensor([0, 1, 2, 3, 5, 6, 7, 100, 4000, 17, 18, 8998], device=DEV)
    length = torch.tensor([8999, 8000, 7777, 1, 2, 3, 4, 5, 4096, 0, 1, 2], device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(4)
    c.rules["history"] = torch.randint(-2, 700, (9003,), generator=gen, device=DEV,
                                       dtype=torch.int32)
    c.rules["history_begin"], c.rules["history_end"] = begin, begin + length
    c.rules["history_split"] = begin + length // 3
    for off in range(4):
        # and the tokens themselves at any place
        whole = torch.cat([c.rules["history"][:off], c.rules["history"]])
        c.rules["history"] = whole[off:]
        y, _, err = C.processed64(c)
        out = rlk.process_logits(c.x, rules(c), real_vocab=v, padded_vocab=v,
                                 out_dtype=torch.float32)
        bound = torch.where(y == -math.inf, 0.0, err + C.H * (y.abs() + err) + C.TINY)
        assert C.worst(out, y, bound) <= 1.0, off


def test_history_bounds_outside_the_tokens():
    """Positions outside the history are not read; an end in front of its begin is no history."""
    n, v = 6, 500
    c = C.make_case(n, v, v, 8, DEV, "penalties")
    total = c.rules["history"].numel()
    big = 2 ** 62
    for name, at in (("begin", [-5, -big, 10, total, total + 7, 20]),
                     ("split", [-9, 3, big, -big, total, 25]),
                     ("end", [4, total + 100, big, big, big, 12])):
        c.rules["history_" + name] = torch.tensor(at, device=DEV)
    y, _, err = C.processed64(c)
    out = rlk.process_logits(c.x, rules(c), real_vocab=v, padded_vocab=v,
                                 out_dtype=torch.float32)
    assert C.worst(out, y, err + C.H * (y.abs() + err)) <= 1.0
    del c.rules["history_split"]  # all of it is generated
    y, _, err = C.processed64(c)
    out = rlk.process_logits(c.x, rules(c), real_vocab=v, padded_vocab=v,
                                 out_dtype=torch.float32)
    assert C.worst(out, y, err + C.H * (y.abs() + err)) <= 1.0


def test_tables_without_an_index():
    """One row for all, one dimension, or a row each."""
    n, v = 5, 3001
    c = C.make_case(n, v, v, 9, DEV, "all")
    for name in ("bias", "allow"):
        del c.rules[name + "_index"]
    bias, allow = c.rules["bias"], c.rules["allow"]
    each = torch.cat([bias, bias])[:n]
    for b, a in ((bias[:1], allow[:1]), (bias[0], allow[0]),
                 (each, torch.cat([allow, allow])[:n])):
        c.rules["bias"], c.rules["allow"] = b, a
        y, _, err = C.processed64(c)
        c.x[:, :v] = torch.where(torch.isfinite(c.x[:, :v].float()), c.x[:, :v], 1.0)
        y, _, err = C.processed64(c)
        out = rlk.process_logits(c.x, rules(c), real_vocab=v, padded_vocab=v,
                                 out_dtype=torch.float32)
        bound = torch.where(y == -math.inf, 0.0, err + C.H * (y.abs() + err) + C.TINY)
        assert C.worst(out, y, bound) <= 1.0


def test_rows_barred_altogether_and_lowest_values():
    """A row without an allowed column: LSE -inf, logp NaN and a gradient of +0.  Logits of the
    type's lowest value, of -inf and of NaN that a grammar bars take part in nothing."""
    n, v = 4, 2500
    c = C.make_case(n, v, v, 10, DEV, "none")
    lowest = torch.finfo(torch.bfloat16).min
    free = torch.zeros(n, 2528, dtype=torch.bool, device=DEV)
    free[1, 7] = free[2, 2499] = free[3, 0] = free[3, 2400] = True
    c.rules = {"allow": C.pack(free), "temperature": torch.full((n,), 0.5, device=DEV)}
    c.x[0, ::3], c.x[0, 1::3], c.x[1, 8:] = math.nan, math.inf, math.nan
    c.x[3, 0] = lowest  # over 0.5: -inf in fp32, beside a finite column
    c.tgt[:] = torch.tensor([5, 7, 2499, 0])
    c.mask[:] = True
    c.x[1, 7], c.x[2, 2499], c.x[3, 2400] = 1.5, lowest / 4, -2.0
    logp, lse = forward(c)
    assert lse[0] == -math.inf and logp[0].isnan()
    assert (lse[1], logp[1]) == (3.0, 0.0)
    assert lse[2] == float(torch.tensor(lowest / 4).bfloat16()) * 2 and logp[2] == 0.0
    assert lse[3] == -4.0 and logp[3] == -math.inf
    d = backward(c, lse, c.g, c.gl)
    assert (bits(d[0]) == 0).all()
    assert (bits(d[~free[:, :v]]) == 0).all()
    # p = 1 in the only column: g (1 - 1) + gl, times 1 / T; gl - g is rounded, and so is its
    # sum with g
    for r, j in ((1, 7), (2, 2499)):
        assert (d[r, j] - 2 * c.gl[r]).abs() <= 2 * C.H * ((c.gl[r] - c.g[r]).abs()
                                                           + 1.01 * c.gl[r].abs())
    assert d[3, 2400] == 2 * (c.gl[3] - c.g[3])
    with pytest.raises(rlk.RlkError) as ei:
        forward(c, validate=True)
    assert ei.value.status == rlk.RLK_ERR_NONFINITE_LSE
    out = rlk.process_logits(c.x, rules(c), real_vocab=v, padded_vocab=v)
    assert (out[~free[:, :v]] == -math.inf).all()


def test_bad_targets_and_rows_that_no_term_reaches():
    n, v, pad = 6, 3000, 3010
    c = C.make_case(n, v, pad, 11, DEV, "all")
    c.mask[:] = True
    c.mask[3] = False
    c.tgt[:] = torch.tensor([1, -1, v, 2 ** 31 - 1, C.IGNORE, 2])
    g, gl = c.g.clone(), torch.zeros_like(c.gl)
    g[5] = 0.0
    c.x[3:] = math.nan  # not read by the gradient
    logp, lse = forward(c)
    assert logp[1].isnan() and logp[2].isnan() and logp[3] == 0 and logp[4] == 0
    d = backward(c, lse, g, gl)
    assert torch.isfinite(d[0]).all() and (d[0] != 0).any()
    assert d[1:3, :v].isnan().all() and (bits(d[1:3, v:]) == 0).all()
    assert (bits(d[3:]) == 0).all()
    for call in (lambda: forward(c, validate=True),
                 lambda: backward(c, lse, g, gl, validate=True)):
        with pytest.raises(rlk.RlkError) as ei:
            call()
        assert ei.value.status == rlk.RLK_ERR_TARGET_RANGE


def test_in_place_and_what_lies_behind():
    n, v, pad = 9, 9001, 9003
    c = C.make_case(n, v, pad, 12, DEV, "all")
    want = rlk.process_logits(c.x, rules(c), real_vocab=v, padded_vocab=pad)
    for dtype in (torch.bfloat16, torch.float32):
        wide = torch.full((n, 9024), 7.0, dtype=dtype, device=DEV)
        got = rlk.process_logits(c.x, rules(c), real_vocab=v, padded_vocab=pad, out=wide,
                                 out_dtype=dtype)
        assert got is wide and (wide[:, pad:] == 7.0).all()
        assert torch.equal(bits(wide[:, :pad].bfloat16()), bits(want))
    x = c.x.clone()
    got = rlk.process_logits(x, rules(c), real_vocab=v, padded_vocab=pad, out=x)
    assert got is x and torch.equal(bits(x[:, :pad]), bits(want))
    assert torch.equal(bits(x[:, pad:]), bits(c.x[:, pad:]))
    # rows of a wider tensor, and only some of its columns
    big = torch.zeros(2 * n, 9032, dtype=torch.bfloat16, device=DEV)
    big[::2, :c.x.shape[1]] = c.x
    part = big[::2, :pad]
    assert torch.equal(bits(rlk.process_logits(part, rules(c), real_vocab=v, padded_vocab=pad)),
                       bits(want))


def test_autograd_sees_what_is_written_in_place():
    """A backward pass that saved the logits refuses them once they are processed in place."""
    c = C.make_case(5, 1000, 1008, 3, DEV, "all")
    for inner in (lambda x: rlk.processed_selected_token_logprob(x, c.tgt, rules(c), c.mask,
                                                                 real_vocab=c.v)[0],
                  lambda x: rlk.selected_token_logprob(x, c.tgt, c.mask, real_vocab=c.v)):
        x = c.x.clone().requires_grad_()
        logp = inner(x)
        logp = logp if isinstance(logp, torch.Tensor) else logp[0]
        g = torch.ones_like(logp)
        torch.autograd.grad(logp, x, g, retain_graph=True)
        with torch.no_grad():
            rlk.process_logits(x, rules(c), real_vocab=c.v, out=x)
        with pytest.raises(RuntimeError, match="inplace"):
            torch.autograd.grad(logp, x, g)


def test_a_row_has_the_same_bits_alone():
    c = C.make_case(40, 20001, 20008, 13, DEV, "all")
    y = rlk.process_logits(c.x, rules(c), real_vocab=c.v, padded_vocab=c.pad)
    logp, lse = forward(c)
    d = backward(c, lse, c.g, c.gl)
    for r in (0, 17, 39):
        o = c.row(r)
        assert torch.equal(bits(rlk.process_logits(o.x, rules(o), real_vocab=c.v,
                                                   padded_vocab=c.pad)), bits(y[r:r + 1]))
        lp, ls = forward(o)
        assert torch.equal(bits(lp), bits(logp[r:r + 1])) and \
            torch.equal(bits(ls), bits(lse[r:r + 1]))
        assert torch.equal(bits(backward(o, ls, o.g, o.gl)), bits(d[r:r + 1]))


def test_without_rules_it_is_the_plain_logp():
    """No rule: the LSE and logp of forward(), but for the order of the sums."""
    c = C.make_case(30, 30001, 30008, 14, DEV, "none")
    a, b = forward(c), rlk.forward(c.x, c.tgt, c.mask, real_vocab=c.v, padded_vocab=c.pad)
    *_, e_logp, e_lse, _ = C.logp64(c)
    assert C.worst(a[0], b[0].double(), 2 * e_logp) <= 1.0
    assert C.worst(a[1], b[1].double(), 2 * e_lse) <= 1.0


def test_autograd():
    c = C.make_case(20, 5000, 5003, 15, DEV, "all")
    x = c.x.clone().requires_grad_(True)
    logp, lse = rlk.processed_selected_token_logprob(x, c.tgt, rules(c), c.mask, real_vocab=c.v,
                                                     padded_vocab=c.pad)
    a, b = forward(c)
    assert torch.equal(bits(logp.detach()), bits(a)) and torch.equal(bits(lse.detach()), bits(b))
    d, = torch.autograd.grad([logp, lse], x, [c.g, c.gl], retain_graph=True)
    want = backward(c, lse.detach(), c.g, c.gl, out_dtype=torch.bfloat16)
    assert d.shape == x.shape and torch.equal(bits(d[:, :c.pad]), bits(want))
    assert (bits(d[:, c.pad:]) == 0).all()
    # one output alone, with an expanded gradient
    d, = torch.autograd.grad(logp.sum(), x, retain_graph=True)
    assert torch.equal(bits(d[:, :c.pad]),
                       bits(backward(c, lse.detach(), torch.ones_like(c.g), None,
                                     out_dtype=torch.bfloat16)))
    with pytest.raises(RuntimeError):  # second derivatives are refused
        first, = torch.autograd.grad(logp.sum(), x, create_graph=True)
        torch.autograd.grad(first.float().sum(), x)
    c.rules["temperature"].mul_(1.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(logp.sum(), x)
    bias = torch.zeros(c.v, device=DEV, requires_grad=True)
    with pytest.raises(ValueError, match="constants"):
        rlk.processed_selected_token_logprob(x, c.tgt, rlk.LogitRules(bias=bias), real_vocab=c.v)


def test_gradient_against_differences():
    """Central differences of the kernel's own logp and LSE, one logit moved by 1/4 up and down
    in steps that bf16 holds: off by 1/6 (1/4)^2 of the third derivative (below (dy/dx)^3 / 8 for
    a softmax: 4^3 / 8) and by two errors of the loss over the step."""
    c = C.make_case(8, 40, 40, 16, DEV, "all", longest=20)
    n, v = 8, c.v
    x = (c.x[:, :v].float().nan_to_num(0, 0, 0).clamp(-6, 6) * 4).round() / 4
    x = torch.where(x.abs() < 0.5, 1.0, x)  # no logit passes 0, where a penalty bends
    c.x[:, :v] = x.bfloat16()
    _, lse = forward(c)
    d = backward(c, lse, c.g, c.gl).double()
    *_, slope, e_logp, e_lse, _ = C.logp64(c)
    weight = c.g.abs().double() + c.gl.abs().double()
    noise = c.g.abs().double() * e_logp + c.gl.abs().double() * e_lse

    def loss(x):
        logp, lse = rlk.processed_forward(x, c.tgt, rules(c), c.mask, real_vocab=v)
        return logp.double() * c.g.double() + lse.double() * c.gl.double()

    for j in range(v):
        up, down = c.x.clone(), c.x.clone()
        up[:, j] += 0.25
        down[:, j] -= 0.25
        got = (loss(up) - loss(down)) / 0.5
        bound = weight * slope[:, j].abs() ** 3 / 8 * 0.25 ** 2 / 6 + 8 * noise + 1e-6
        assert ((got - d[:, j]).abs() <= bound).all(), j


def test_no_rows():
    x = torch.zeros(0, 104, dtype=torch.bfloat16, device=DEV)
    t = torch.zeros(0, dtype=torch.int32, device=DEV)
    f = torch.zeros(0, device=DEV)
    r = rlk.LogitRules(temperature=f)
    assert rlk.process_logits(x, r, real_vocab=100).shape == (0, 104)
    logp, lse = rlk.processed_forward(x, t, r, real_vocab=100)
    assert logp.shape == lse.shape == (0,)
    assert rlk.processed_backward(x, t, r, None, lse, f, real_vocab=100).shape == (0, 104)
    one = torch.zeros(1, 104, dtype=torch.bfloat16, device=DEV)
    empty = rlk.LogitRules(repetition=torch.full((1,), 2.0, device=DEV), history=t,
                           history_begin=torch.zeros(1, dtype=torch.int64, device=DEV),
                           history_end=torch.ones(1, dtype=torch.int64, device=DEV))
    assert (rlk.process_logits(one, empty, real_vocab=104) == 0).all()
