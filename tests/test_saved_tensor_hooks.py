"""Hooks on saved tensors (offloading them to host memory, for instance) hand a backward pass other
tensors than were saved, in another layout; gradients are those without hooks."""
from __future__ import annotations

import pytest
import torch
from torch.autograd.graph import save_on_cpu, saved_tensors_hooks

import vocab_selected_token_amd as rlk
from tests import process_cases as C
from tests.test_host_streams import BF16, K, N, streams  # noqa: F401 (a fixture)


def turned(t):
    """A copy whose last dimension is not the one of unit stride."""
    return t.t().contiguous().t() if t.dim() == 2 else t.clone()


COPIES = {"contiguous": lambda t: t.clone(memory_format=torch.contiguous_format), "turned": turned}


@pytest.mark.parametrize("copy", COPIES)
@pytest.mark.parametrize("v", [96, 101])
def test_rows_are_read_where_they_lie(copy, v, streams, monkeypatch):  # noqa: F811
    """(no GPU) The gradient's call is given rows as far apart as it is told, of a buffer that
    holds them all, and the rules as they were saved."""
    calls = []
    monkeypatch.setattr(rlk, "rlk_logp_processed_bwd", lambda *a: calls.append(a))
    for width in ((v + 7) // 8 * 8, 128):
        wide = torch.arange(N * width).view(N, width).remainder(250).to(torch.bfloat16)
        x = wide[:, :v].requires_grad_()
        temperature, bias = torch.full((N,), 2.0), torch.zeros(3, 2 * v)[:, :v]
        index = torch.zeros(N, dtype=torch.int32)
        rules = rlk.LogitRules(temperature=temperature, bias=bias, bias_index=index)
        targets = torch.zeros(N, dtype=torch.int32)
        with saved_tensors_hooks(COPIES[copy], lambda t: t):
            logp, _ = rlk.processed_selected_token_logprob(x, targets, rules, real_vocab=v)
        temperature.fill_(7.0)
        torch.autograd.grad(logp.sum(), x)
        desc, logits, struct, *_ = calls.pop()
        assert logits.stride() == (desc.ld_logits, 1) and desc.ld_logits % 8 == 0
        assert torch.equal(logits, x)
        assert logits.untyped_storage().nbytes() >= 2 * (N - 1) * desc.ld_logits + 2 * v
        assert struct.temperature != temperature.data_ptr()  # (the 2.0 that was saved)
        assert struct.bias_rows == 3 and struct.ld_bias >= v


@pytest.mark.parametrize("copy", COPIES)
def test_products_are_given_contiguous_tensors(copy, streams, monkeypatch):  # noqa: F811
    calls = []
    monkeypatch.setattr(rlk, "rlk_linear_bwd", lambda *a: calls.append(a))
    x = torch.zeros(N, K, **BF16).requires_grad_()
    w = torch.zeros(77, K, **BF16).requires_grad_()
    with saved_tensors_hooks(COPIES[copy], lambda t: t):
        y = rlk.head_linear(x, w, activation="silu")
    torch.autograd.grad(y, (x, w), torch.zeros_like(y))
    (_, *tensors), = calls
    assert len(tensors) > 3 and all(t.is_contiguous() for t in tensors[:3])


@pytest.mark.parametrize("copy", COPIES)
def test_the_lmhead_is_given_contiguous_tensors(copy, streams, monkeypatch):  # noqa: F811
    calls = []
    monkeypatch.setattr(rlk, "rlk_logp_fused_lmhead_bwd", lambda *a: calls.append(a))
    x = torch.zeros(N, K, **BF16).requires_grad_()
    w = torch.zeros(512, K, **BF16).requires_grad_()
    with saved_tensors_hooks(COPIES[copy], lambda t: t):
        logp, _ = rlk.lmhead_selected_token_logprob(x, w, torch.zeros(N, dtype=torch.int32),
                                                    real_vocab=500, num_vocab_tiles=2)
    torch.autograd.grad(logp.sum(), (x, w))
    (_, hidden, weight, *_), = calls
    assert hidden.is_contiguous() and weight.is_contiguous()


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("hooks", ["cpu", *COPIES])
@pytest.mark.parametrize("n, v, pad", [(1, 77, 80), (9, 3001, 3005), (60, 1000, 1000)])
def test_gradients(hooks, n, v, pad):
    print(f"case {hooks} {n} {v} {pad}", flush=True)
    dev = torch.device("cuda")
    c = C.make_case(n, v, pad, 41, dev)
    h = torch.randn(n, 64, device=dev).bfloat16()
    w = (torch.randn(pad, 64, device=dev) / 8).bfloat16()
    leaves = [h.requires_grad_(), w.requires_grad_()]

    def forward():
        rules = rlk.LogitRules(**{k: t.clone() for k, t in c.rules.items()})
        z = rlk.head_linear(h, w, activation="silu")
        logp, lse = rlk.processed_selected_token_logprob(z, c.tgt, rules, c.mask, real_vocab=v)
        return rules, (logp * c.g).sum() + (lse * c.gl).sum()

    want = torch.autograd.grad(forward()[1], leaves)
    with save_on_cpu() if hooks == "cpu" else \
            saved_tensors_hooks(COPIES[hooks], lambda t: t):
        rules, loss = forward()
    for t in rules.tensors:  # (what was saved are copies)
        t.zero_()
    got = torch.autograd.grad(loss, leaves)
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
