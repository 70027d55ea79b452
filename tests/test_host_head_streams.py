"""Where the logit rules' and the dense products' conveniences take memory for a call on another
stream (no GPU; the stand-ins of tests/test_host_streams.py)."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests.test_host_streams import K, N, V, check, streams  # noqa: F401 (a fixture)

RULES = rlk.LogitRules(temperature=torch.ones(N))
SAVED = torch.zeros(N, V, dtype=torch.float16)
CALLS = {
    "process_logits": lambda i, **kw: rlk.process_logits(i["x"], RULES, real_vocab=V, **kw),
    "processed_forward": lambda i, **kw: rlk.processed_forward(i["x"], i["t"], RULES,
                                                               real_vocab=V, **kw),
    "processed_backward": lambda i, **kw: rlk.processed_backward(
        i["x"], i["t"], RULES, None, i["f"], i["f"], real_vocab=V, **kw),
    "linear_forward": lambda i, **kw: rlk.linear_forward(i["h"], i["w"], activation="silu",
                                                         save=True, **kw),
    "linear_backward": lambda i, **kw: rlk.linear_backward(
        i["h"], i["w"], i["x"], SAVED, activation="silu", want_bias=True, **kw),
    "lmhead_logits": lambda i, **kw: rlk.lmhead_logits(i["h"], i["w"], real_vocab=V, **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_launch_stream(name, streams):  # noqa: F811
    assert K % 64 == 0
    check(CALLS[name], streams)
