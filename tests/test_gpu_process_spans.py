"""The logit rules where a block takes four spans of a row (many rows): grammars, biases and
histories longer than what a block keeps of them, against the formulas in 64 bits and against the
same rows alone, whose blocks take one span each.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import process_cases as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
SPAN = 8192          # columns of a span
MANY_BLOCKS = 16384  # spans of all rows from which a block takes four
HELD = 4096          # tokens of a history that a block keeps


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def calls(c):
    r = rlk.LogitRules(**c.rules)
    kw = dict(real_vocab=c.v, padded_vocab=c.pad)
    out = {"bf16": rlk.process_logits(c.x, r, **kw),
           "fp32": rlk.process_logits(c.x, r, out_dtype=torch.float32, **kw)}
    out["logp"], out["lse"] = rlk.processed_forward(c.x, c.tgt, r, c.mask, **kw)
    out["grad"] = rlk.processed_backward(c.x, c.tgt, r, c.mask, out["lse"], c.g, c.gl,
                                         out_dtype=torch.bfloat16, **kw)
    return out


# the last block of a row takes one, two, three and four spans
@pytest.mark.parametrize("n, v, pad", [(3400, 33001, 33008), (2800, 49001, 49003),
                                       (2400, 57001, 57344), (2100, 65500, 65536)])
def test_four_spans_a_block(n, v, pad):
    print(f"case {n} {v} {pad}", flush=True)
    assert n * -(-v // SPAN) >= MANY_BLOCKS
    c = C.make_case(n, v, pad, n, DEV, "all", longest=2 * HELD + 1000)
    got = calls(c)
    lengths = c.rules["history_end"] - c.rules["history_begin"]
    index = c.rules["allow_index"]
    barred = (index >= 0) & (index < 4)
    assert int(lengths.max()) > 2 * HELD
    rows = {int(lengths.argmax()), 0, n - 1, int((lengths * barred).argmax()),
            int(((lengths > HELD) & ~barred).int().argmax()), int(barred.int().argmax()),
            n // 2, n // 3}
    assert any(barred[r] for r in rows) and any(not barred[r] for r in rows)
    for r in sorted(rows):
        one = c.row(r)
        alone = calls(one)
        for k, t in alone.items():
            assert torch.equal(bits(t), bits(got[k][r:r + 1])), (k, r)
        y, _, err = C.processed64(one)
        for k, half in (("bf16", C.HALF_BF16), ("fp32", C.H)):
            bound = err + half * (torch.where(y == -torch.inf, 0.0, y).abs() + err)
            bound = torch.where(y == -torch.inf, 0.0, bound + C.TINY)
            assert C.worst(alone[k][:, :v], y, bound) <= 1.0, (k, r)
            assert (alone[k][:, v:] == -torch.inf).all()
        logp, lse, _, _, e_logp, e_lse, _ = C.logp64(one)
        assert C.worst(alone["logp"], logp, e_logp) <= 1.0, r
        assert C.worst(alone["lse"], lse, e_lse) <= 1.0, r
        assert C.worst(alone["grad"], *C.gradient64(one, one.g, one.gl, C.HALF_BF16)) <= 1.0, r
