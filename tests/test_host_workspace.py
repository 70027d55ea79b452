"""A workspace of the caller's that a call cannot use is refused before anything is enqueued (no GPU;
the stand-ins of tests/test_host_streams.py)."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import test_host_head_streams as head
from tests.test_host_streams import LMHEAD, LOGITS, inputs, streams  # noqa: F401 (a fixture)

CALLS = {name: call for name, call in {**LMHEAD, **LOGITS, **head.CALLS}.items()
         if name not in ("quantize_fp8", "quantize_fp8_weight", "lmhead_logits_fp8",
                         "process_logits", "linear_forward", "lmhead_logits")}


@pytest.mark.parametrize("name", CALLS)
def test_workspaces(name, streams, monkeypatch):  # noqa: F811
    size, calls = 1 << 16, []

    class Library(type(rlk._lib)):
        def __getattr__(self, entry):
            if entry.endswith("workspace_bytes"):
                return lambda *a: size
            return lambda *a: calls.append(entry) or 0

    monkeypatch.setattr(rlk, "_lib", Library())
    call, i = CALLS[name], inputs()
    for ws, error, match in ((torch.empty(size, dtype=torch.uint8, device="meta"), ValueError,
                              "workspace is on meta"),
                             (torch.empty(2 * size, dtype=torch.uint8)[::2], ValueError,
                              "contiguous"),
                             (bytearray(size), TypeError, "torch.Tensor")):
        with pytest.raises(error, match=match):
            call(i, workspace=ws)
        assert not calls
    call(i, workspace=torch.empty(size, dtype=torch.uint8))
    call(i, workspace=torch.empty(size // 4))  # any type will do
    assert calls
