"""What the dense products return: whole rows, padded to 8 columns, and a tensor of its own (no GPU; the
stand-ins of tests/test_host_streams.py)."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests.test_host_streams import BF16, K, N, streams  # noqa: F401 (a fixture)


@pytest.mark.parametrize("n", [1, 8, 77, 80])
def test_a_result_can_be_changed_in_place(n, streams):  # noqa: F811
    """With any number of outputs: autograd saves the inputs, not the result."""
    x, w = torch.zeros(N, K, **BF16).requires_grad_(), torch.zeros(n, K, **BF16)
    for make in (lambda: rlk.head_linear(x, w, activation="silu"),
                 lambda: rlk.linear_forward(x.detach(), w)[0],
                 lambda: rlk.lmhead_logits(x.detach(), w, real_vocab=n)):
        y = make()
        assert y.shape == (N, n) and y.stride() == ((n + 7) // 8 * 8, 1)
        assert y.untyped_storage().nbytes() == N * y.stride(0) * 2
        y.zero_().add_(1.0)
        assert (y == 1.0).all()
    y = rlk.head_linear(x, w, activation="silu")
    y += torch.ones_like(y)
    y[0] = 3.0
    g, = torch.autograd.grad(y.sum(), x)
    assert g.shape == x.shape
