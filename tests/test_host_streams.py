"""Where the conveniences take memory for a call on another stream than the current one (no
GPU: the library and torch's streams are stood in for).

Memory for work on a stream has to come from that stream's pool: a block that the current
stream's work still uses may be handed out again on the current stream alone.  What is
returned is read on the current stream, so it is recorded there."""
from __future__ import annotations

import contextlib

import pytest
import torch

import vocab_selected_token_amd as rlk

N, K, V = 6, 128, 512
BF16 = dict(dtype=torch.bfloat16)


class Stream:
    def __init__(self, name, handle):
        self.name, self.cuda_stream = name, handle


class Library:
    """Every call succeeds; sizes are 64 KB."""

    def __getattr__(self, name):
        return (lambda *a: 1 << 16) if name.endswith("workspace_bytes") else (lambda *a: 0)


CURRENT, SIDE = Stream("current", 0x100), Stream("side", 0x200)


@pytest.fixture
def streams(monkeypatch):
    """What was allocated on which stream, and which tensors were recorded where."""
    seen = {"on": [CURRENT], "made": [], "recorded": []}

    @contextlib.contextmanager
    def on(stream):
        seen["on"].append(stream)
        yield
        seen["on"].pop()

    def watched(make):
        def call(*a, **kw):
            t = make(*a, **kw)
            seen["made"].append((seen["on"][-1], t))
            return t
        return call

    for name in ("empty", "empty_like", "empty_strided", "zeros", "zeros_like"):
        monkeypatch.setattr(torch, name, watched(getattr(torch, name)))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: seen["recorded"].append((t, s)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: seen["on"][-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(rlk, "_check_device", lambda *a, **kw: None)
    monkeypatch.setattr(rlk, "_stream", lambda s: 0)
    monkeypatch.setattr(rlk, "_torch_stream", lambda s, device: s, raising=False)
    monkeypatch.setattr(rlk, "_lib", Library())
    return seen


def inputs():
    return dict(h=torch.zeros(N, K, **BF16), w=torch.zeros(V, K, **BF16),
                x=torch.zeros(N, V, **BF16), t=torch.zeros(N, dtype=torch.int32),
                f=torch.zeros(N), wq=torch.zeros(V, K, dtype=torch.float8_e4m3fn),
                ws=torch.ones(V // 128, 1))


LMHEAD = {
    "fused_lmhead": lambda i, **kw: rlk.fused_lmhead(i["h"], i["w"], i["t"], real_vocab=V,
                                                     num_vocab_tiles=2, **kw),
    "fused_lmhead_backward": lambda i, **kw: rlk.fused_lmhead_backward(
        i["h"], i["w"], i["t"], None, i["f"], i["f"], real_vocab=V, **kw),
    "quantize_fp8": lambda i, **kw: rlk.quantize_fp8(i["h"], **kw),
    "quantize_fp8_weight": lambda i, **kw: rlk.quantize_fp8(i["w"], 128, **kw),
    "lmhead_logits_fp8": lambda i, **kw: rlk.lmhead_logits_fp8(i["h"], i["wq"], i["ws"],
                                                               real_vocab=V, **kw),
    "fused_lmhead_fp8": lambda i, **kw: rlk.fused_lmhead_fp8(
        i["h"], i["wq"], i["ws"], i["t"], real_vocab=V, num_vocab_tiles=2, **kw),
}


def check(call, seen):
    i = inputs()
    seen["made"].clear()
    out = call(i, stream=SIDE)
    assert seen["made"], "nothing was allocated"
    assert all(s is SIDE for s, _ in seen["made"])
    out = out if isinstance(out, tuple) else (out,)
    recorded = {t.untyped_storage().data_ptr() for t, s in seen["recorded"] if s is CURRENT}
    assert all(t.untyped_storage().data_ptr() in recorded for t in out)
    # on the current stream nothing changes hands
    seen["recorded"].clear()
    seen["made"].clear()
    call(i)
    call(i, stream=CURRENT)
    assert seen["made"] and all(s is CURRENT for s, _ in seen["made"])
    assert not seen["recorded"]


@pytest.mark.parametrize("name", LMHEAD)
def test_lmhead_memory_comes_from_the_launch_stream(name, streams):
    check(LMHEAD[name], streams)


LOGITS = {
    "forward": lambda i, **kw: rlk.forward(i["x"], i["t"], real_vocab=V, **kw),
    "backward": lambda i, **kw: rlk.backward(i["x"], i["t"], None, i["f"], i["f"], real_vocab=V,
                                             **kw),
    "forward_ex": lambda i, **kw: rlk.forward_ex(i["x"], i["t"], real_vocab=V, **kw),
    "backward_ex": lambda i, **kw: rlk.backward_ex(i["x"], i["t"], None, i["f"], i["f"], i["f"],
                                                   real_vocab=V, **kw),
    "forward_backward": lambda i, **kw: rlk.forward_backward(i["x"], i["t"], None, i["f"],
                                                             real_vocab=V, **kw),
    "forward_backward_ex": lambda i, **kw: rlk.forward_backward_ex(i["x"], i["t"], None, i["f"],
                                                                   real_vocab=V, **kw),
}


@pytest.mark.parametrize("name", LOGITS)
def test_logits_memory_comes_from_the_launch_stream(name, streams):
    check(LOGITS[name], streams)
