"""Calls on a stream of their own while the current stream is busy: what the busy stream still
reads from memory that was freed in the meantime stays, and so do the call's results.  Needs
an MI355X."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import lmhead_cases as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
N, K, V = 300, 256, 2900


class Handle:
    """A stream that torch did not make: a handle."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.fixture(scope="module")
def inputs():
    c = C.make_case(N, K, V, V, 7, DEV)
    wq, ws = rlk.quantize_fp8(c.w, 128)
    _, lse = rlk.fused_lmhead(c.h, c.w, c.tgt, c.mask, real_vocab=V, num_vocab_tiles=7)
    return c, wq, ws, lse


LMHEAD = {
    "fused_lmhead": lambda c, wq, ws, lse, **kw: rlk.fused_lmhead(
        c.h, c.w, c.tgt, c.mask, real_vocab=V, num_vocab_tiles=7, **kw),
    "fused_lmhead_backward": lambda c, wq, ws, lse, **kw: rlk.fused_lmhead_backward(
        c.h, c.w, c.tgt, c.mask, lse, c.g, c.gl, real_vocab=V, **kw),
    "quantize_fp8": lambda c, wq, ws, lse, **kw: rlk.quantize_fp8(c.w, 128, **kw),
    "lmhead_logits_fp8": lambda c, wq, ws, lse, **kw: rlk.lmhead_logits_fp8(
        c.h, wq, ws, real_vocab=V, **kw),
    "fused_lmhead_fp8": lambda c, wq, ws, lse, **kw: rlk.fused_lmhead_fp8(
        c.h, wq, ws, c.tgt, c.mask, real_vocab=V, num_vocab_tiles=7, **kw),
}


def raw(out):
    return [t.contiguous().view(torch.uint8).clone()
            for t in (out if isinstance(out, tuple) else (out,))]


def check(call, inputs):
    """The current stream: a delay, then copies of tensors of every size a call may take, which
    are freed as soon as the copies are queued.  The side stream does not wait."""
    want = raw(call(*inputs))
    side = torch.cuda.Stream()
    sizes = [1 << p for p in range(9, 26)] * 2
    for stream in (side, Handle(side)):
        torch.cuda.synchronize()
        held = [torch.full((s,), 0x5a, dtype=torch.uint8, device=DEV) for s in sizes]
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)  # some 50 ms
        copies = [h.clone() for h in held]
        del held
        outs = [call(*inputs, stream=stream) for _ in range(3)]
        side.synchronize()
        busy = not torch.cuda.current_stream().query()
        torch.cuda.current_stream().wait_stream(side)
        got = [raw(o) for o in outs]
        del outs  # back to the side stream's pool, while the current stream reads them
        call(*inputs, stream=stream)
        torch.cuda.synchronize()
        assert busy, "the delay ended before the calls did: nothing was shown"
        for o in got:
            assert all(torch.equal(a, b) for a, b in zip(o, want))
        assert all((c == 0x5a).all() for c in copies)


@pytest.mark.parametrize("name", LMHEAD)
def test_lmhead_calls_beside_a_busy_stream(name, inputs):
    print(f"case {name}", flush=True)
    check(LMHEAD[name], inputs)


LOGITS = {
    "forward": lambda x, t, m, f, **kw: rlk.forward(x, t, m, real_vocab=V, **kw),
    "backward": lambda x, t, m, f, **kw: rlk.backward(x, t, m, f, f, real_vocab=V, **kw),
    "forward_ex": lambda x, t, m, f, **kw: rlk.forward_ex(x, t, m, real_vocab=V, **kw),
    "backward_ex": lambda x, t, m, f, **kw: rlk.backward_ex(x, t, m, f, f, f, real_vocab=V, **kw),
    "forward_backward": lambda x, t, m, f, **kw: rlk.forward_backward(x, t, m, f, real_vocab=V,
                                                                      **kw),
    "forward_backward_ex": lambda x, t, m, f, **kw: rlk.forward_backward_ex(
        x, t, m, f, real_vocab=V, **kw),
}


@pytest.mark.parametrize("name", LOGITS)
def test_logits_calls_beside_a_busy_stream(name, inputs):
    print(f"case {name}", flush=True)
    c, wq, ws, lse = inputs
    x = rlk.lmhead_logits_fp8(c.h, wq, ws, real_vocab=V, padded_vocab=V + 4)
    torch.cuda.synchronize()
    check(LOGITS[name], (x, c.tgt, c.mask, lse))
