"""The handle of the current stream, with and without torch's direct call for it (no GPU)."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

import vocab_selected_token_amd as rlk


@pytest.mark.parametrize("direct", [True, False])
def test_current_stream(direct, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(rlk, "_raw_stream", (lambda device: 70 + device) if direct else None)
    assert rlk._stream(None) == (73 if direct else 77)
    assert rlk._stream(SimpleNamespace(cuda_stream=5)) == 5
