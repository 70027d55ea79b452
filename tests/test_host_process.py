"""Refusals of the logit rules' entry points, and the plain form that their GPU tests are held to
against differences (no GPU: nothing launches a kernel)."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import process_cases as C
from tests.test_host_fp8 import FakeTensor, NoStream, refused

A, WS = FakeTensor(0x10000000), FakeTensor(0x20000000)
PTR = 0x10000000


def desc(**kw):
    return rlk.make_desc(**{**dict(num_tokens=8, real_vocab=1000, padded_vocab=1024,
                                   ld_logits=1024, num_vocab_tiles=4), **kw})


def rules(**kw):
    s = rlk.rlk_logit_rules()
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def process(d=None, r=rules(), x=A, out=WS, ld=1024, dtype=rlk.RLK_DTYPE_BF16):
    rlk.rlk_logits_process(desc() if d is None else d, x, r, out, ld, dtype, stream=NoStream())


def forward(d=None, r=rules(), x=A, tgt=A, logp=A, lse=A, ws=WS):
    rlk.rlk_logp_processed_fwd(desc() if d is None else d, x, r, tgt, None, logp, lse, ws,
                               stream=NoStream())


def backward(d=None, r=rules(), x=A, tgt=A, lse=A, g=A, gl=A, out=WS, ld=1024,
             dtype=rlk.RLK_DTYPE_BF16, ws=WS):
    rlk.rlk_logp_processed_bwd(desc() if d is None else d, x, r, tgt, None, lse, g, gl, out, ld,
                               dtype, ws, stream=NoStream())


HISTORY = dict(history=PTR, history_len=10, history_begin=PTR, history_end=PTR)


@pytest.mark.parametrize("call", [process, forward, backward])
@pytest.mark.parametrize("kw, code", [
    (dict(d=desc(num_tokens=-1)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(real_vocab=0)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(d=desc(ld_logits=1028)), rlk.RLK_ERR_ALIGNMENT),
    (dict(d=desc(num_vocab_tiles=0)), rlk.RLK_ERR_BAD_TILING),
    # column numbers of the last block would pass 2^31
    (dict(d=desc(padded_vocab=(1 << 31) - 8, ld_logits=(1 << 31) - 8)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(x=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(x=FakeTensor(PTR + 8)), rlk.RLK_ERR_ALIGNMENT),
    (dict(r=None), rlk.RLK_ERR_NULL_POINTER),
    (dict(r=rules(temperature=PTR + 2)), rlk.RLK_ERR_ALIGNMENT),
    (dict(r=rules(**{**HISTORY, "history_len": -1})), rlk.RLK_ERR_BAD_SHAPE),
    (dict(r=rules(**{**HISTORY, "history_len": 1 << 31})), rlk.RLK_ERR_BAD_SHAPE),
    (dict(r=rules(**{**HISTORY, "history_begin": None})), rlk.RLK_ERR_NULL_POINTER),
    (dict(r=rules(**{**HISTORY, "history_end": None})), rlk.RLK_ERR_NULL_POINTER),
    (dict(r=rules(**{**HISTORY, "history_end": PTR + 4})), rlk.RLK_ERR_ALIGNMENT),
    (dict(r=rules(**HISTORY, history_split=PTR + 4)), rlk.RLK_ERR_ALIGNMENT),
    (dict(r=rules(bias=PTR, bias_rows=1, ld_bias=999)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(r=rules(bias=PTR, bias_rows=0, ld_bias=1000)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(r=rules(bias=PTR, bias_rows=3, ld_bias=1000)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(r=rules(bias=PTR + 2, bias_rows=1, ld_bias=1000)), rlk.RLK_ERR_ALIGNMENT),
    (dict(r=rules(allow=PTR, allow_rows=1, ld_allow=31)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(r=rules(allow=PTR, allow_rows=7, ld_allow=32)), rlk.RLK_ERR_BAD_SHAPE),
    (dict(r=rules(allow=PTR, allow_rows=7, ld_allow=32, allow_index=PTR + 1)),
     rlk.RLK_ERR_ALIGNMENT),
])
def test_calls_refuse(call, kw, code):
    refused(call, code, **kw)


def test_process_refuses():
    refused(process, rlk.RLK_ERR_BAD_SHAPE, d=desc(validate=True))
    refused(process, rlk.RLK_ERR_DTYPE, dtype=2)
    refused(process, rlk.RLK_ERR_BAD_SHAPE, ld=1016)
    refused(process, rlk.RLK_ERR_ALIGNMENT, ld=1028)
    refused(process, rlk.RLK_ERR_NULL_POINTER, out=None)
    refused(process, rlk.RLK_ERR_ALIGNMENT, out=FakeTensor(PTR + 8))
    refused(process, rlk.RLK_ERR_BAD_SHAPE, out=A, dtype=rlk.RLK_DTYPE_F32)
    refused(process, rlk.RLK_ERR_BAD_SHAPE, out=A, ld=1032)
    process(d=desc(num_tokens=0), x=None, out=None)


def test_logp_refuses():
    for call in (forward, backward):
        refused(call, rlk.RLK_ERR_NULL_POINTER, tgt=None)
        refused(call, rlk.RLK_ERR_NULL_POINTER, lse=None)
        refused(call, rlk.RLK_ERR_WORKSPACE, ws=None)
        refused(call, rlk.RLK_ERR_ALIGNMENT, ws=FakeTensor(PTR + 16))
        refused(call, rlk.RLK_ERR_ALIGNMENT, tgt=FakeTensor(PTR + 2))
    need = rlk.rlk_logp_processed_workspace_bytes(desc())
    assert need == 256 + 3 * 256  # 8 rows: one piece each, and the target's logit
    refused(forward, rlk.RLK_ERR_WORKSPACE, ws=FakeTensor(0x20000000, need - 1))
    refused(backward, rlk.RLK_ERR_WORKSPACE, ws=FakeTensor(0x20000000, 255))
    refused(backward, rlk.RLK_ERR_NULL_POINTER, g=None, gl=None)
    refused(backward, rlk.RLK_ERR_BAD_SHAPE, out=A)
    refused(backward, rlk.RLK_ERR_BAD_SHAPE, ld=1016)
    refused(backward, rlk.RLK_ERR_DTYPE, dtype=7)
    forward(d=desc(num_tokens=0), x=None, tgt=None, logp=None, lse=None, ws=None)
    backward(d=desc(num_tokens=0), x=None, tgt=None, lse=None, g=None, gl=None, out=None, ws=None)
    assert rlk.rlk_logp_processed_workspace_bytes(desc(real_vocab=0)) == 0


def test_rules_check_their_tensors():
    n, v = 4, 100
    f, i = torch.ones(n), torch.zeros(n, dtype=torch.int64)
    tokens = torch.zeros(9, dtype=torch.int32)
    with pytest.raises(TypeError, match="float32"):
        rlk.LogitRules(repetition=f.double())
    with pytest.raises(TypeError, match="torch.Tensor"):
        rlk.LogitRules(temperature=0.7)
    with pytest.raises(ValueError, match="contiguous"):
        rlk.LogitRules(presence=torch.ones(n, 2)[:, 0])
    with pytest.raises(ValueError, match="other rules"):
        rlk.LogitRules(presence=f, frequency=torch.ones(n + 1))
    with pytest.raises(TypeError, match="history_begin"):
        rlk.LogitRules(history=tokens)
    with pytest.raises(TypeError, match="need a history"):
        rlk.LogitRules(history_begin=i)
    with pytest.raises(TypeError, match="int32"):
        rlk.LogitRules(history=tokens.long(), history_begin=i, history_end=i)
    with pytest.raises(TypeError, match="int64"):
        rlk.LogitRules(history=tokens, history_begin=i.int(), history_end=i)
    with pytest.raises(ValueError, match="other rules"):
        rlk.LogitRules(history=tokens, history_begin=i, history_end=i[:2])
    with pytest.raises(TypeError, match="needs a bias"):
        rlk.LogitRules(bias_index=i.int())
    with pytest.raises(TypeError, match="needs allow"):
        rlk.LogitRules(allow_index=i.int())
    with pytest.raises(TypeError, match="float32"):
        rlk.LogitRules(bias=f.bfloat16())
    with pytest.raises(ValueError, match="without an index"):
        rlk.LogitRules(temperature=f, bias=torch.zeros(3, v))
    with pytest.raises(ValueError, match="column stride"):
        rlk.LogitRules(bias=torch.zeros(v, 3).t())
    with pytest.raises(ValueError, match="do not overlap"):
        rlk.LogitRules(bias=torch.zeros(1, v).expand(3, v), bias_index=i.int())
    with pytest.raises(TypeError, match="int32"):
        rlk.LogitRules(allow=torch.zeros(1, 4, dtype=torch.int64))
    assert rlk.LogitRules().rows is None
    r = rlk.LogitRules(bias=torch.zeros(v), allow=torch.zeros(2, 4, dtype=torch.int32),
                       allow_index=i.int())
    assert r.rows == n and r.struct.bias_rows == 1 and r.struct.allow_rows == 2


def test_conveniences_check_their_tensors():
    n, v = 4, 100
    x = torch.zeros(n, 104, dtype=torch.bfloat16)
    t = torch.zeros(n, dtype=torch.int32)
    f = torch.ones(n)
    r = rlk.LogitRules(temperature=f)
    for call in (lambda x, r=r, **kw: rlk.process_logits(x, r, **{"real_vocab": v, **kw}),
                 lambda x, r=r, **kw: rlk.processed_forward(x, t, r, **{"real_vocab": v, **kw}),
                 lambda x, r=r, **kw: rlk.processed_backward(x, t, r, None, f, f,
                                                             **{"real_vocab": v, **kw}),
                 lambda x, r=r, **kw: rlk.processed_selected_token_logprob(
                     x, t, r, **{"real_vocab": v, **kw})):
        with pytest.raises(TypeError, match="bfloat16"):
            call(x.float())
        with pytest.raises(ValueError, match="exceeds"):
            call(x, padded_vocab=105)
        with pytest.raises(ValueError, match="positive"):
            call(x, real_vocab=0)
        with pytest.raises((TypeError, ValueError), match="LogitRules|GPU memory"):
            call(x, r={})
        with pytest.raises(ValueError, match="GPU memory|rows"):
            call(x)
    with pytest.raises(TypeError, match="LogitRules"):
        rlk.process_logits(x, None, real_vocab=v)
    with pytest.raises(ValueError, match="3 rows|4"):
        rlk.process_logits(x, rlk.LogitRules(temperature=f[:3]), real_vocab=v)
    with pytest.raises(ValueError, match="bias has"):
        rlk.process_logits(x, rlk.LogitRules(bias=torch.zeros(99)), real_vocab=v)
    with pytest.raises(ValueError, match="words"):
        rlk.process_logits(x, rlk.LogitRules(allow=t[:3]), real_vocab=v)
    with pytest.raises(ValueError, match="out_dtype"):
        rlk.process_logits(x, r, real_vocab=v, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="out must"):
        rlk.process_logits(x, r, real_vocab=v, out=x.float())
    with pytest.raises(ValueError, match="out must"):
        rlk.process_logits(x, r, real_vocab=v, out=x[:, :96])
    with pytest.raises(TypeError, match="at least one"):
        rlk.processed_backward(x, t, r, None, f, real_vocab=v)
    with pytest.raises(TypeError, match="lse"):
        rlk.processed_backward(x, t, r, None, None, f, real_vocab=v)


def test_out_that_requires_a_gradient_is_refused():
    x = torch.zeros(4, 104, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="requires a gradient"):
        rlk.process_logits(x, rlk.LogitRules(), real_vocab=100, out=x)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU memory"):
        rlk.process_logits(x, rlk.LogitRules(), real_vocab=100, out=x)


@pytest.mark.parametrize("kind", C.KINDS)
def test_the_formula_against_differences(kind):
    """dx of the plain form against central differences of its logp and LSE, in 64 bits: the
    third derivative of either is below (dy/dx)^3 < 20, so a step of 2^-8 is off by less than
    20/6 2^-16 times the weights (1 + |g|, |gl| < 8); no logit lies within a step of 0, where a
    penalty bends."""
    c = C.make_case(5, 70, 75, 3, "cpu", kind, longest=30)
    near = c.x[:, :c.v].float().abs() < 2.0 ** -7
    c.x[:, :c.v] = torch.where(near, torch.tensor(0.5).bfloat16(), c.x[:, :c.v])
    want, _ = C.gradient64(c, c.g, c.gl, 0.0)

    def loss(x):
        logp, lse, *_ = C.logp64(C.Case(x, c.v, c.pad, c.rules, c.tgt, c.mask, c.g, c.gl))
        return logp * c.g.double() + lse * c.gl.double()

    step = 2.0 ** -8
    x = torch.where(torch.isfinite(c.x.double()), c.x.double(), 0.0)
    for j in range(0, c.v, 3):
        up, down = x.clone(), x.clone()
        up[:, j] += step
        down[:, j] -= step
        got = (loss(up) - loss(down)) / (2 * step)
        assert (got - want[:, j]).abs().max() < 20 / 6 * step ** 2 * 8, j
