"""Forward-mode differentiation is refused by every differentiable call: none returns a result
without its tangent."""
from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad

import vocab_selected_token_amd as rlk

N, K, V = 5, 64, 24


def tensors(device):
    def ones(*shape):
        return torch.ones(shape, dtype=torch.bfloat16, device=device)
    return {"x": ones(N, K), "weight": ones(V, K), "bias": ones(V), "residual": ones(N, V)}


def refuses(call, inputs):
    for name, t in inputs.items():
        for grad in (True, False):
            with forward_ad.dual_level(), torch.set_grad_enabled(grad):
                dual = forward_ad.make_dual(t, torch.ones_like(t))
                with pytest.raises(NotImplementedError, match="jvp"):
                    call(**{**inputs, name: dual})


def head_linear(**kw):
    return rlk.head_linear(kw.pop("x"), kw.pop("weight"), **kw)


def test_head_linear_takes_no_way_around_torch(monkeypatch):
    """(no GPU: the product is a stand-in)"""
    ways = []

    def product(x, w, *args):
        ways.append("product")
        return torch.zeros(N, V), None

    monkeypatch.setattr(rlk, "_check_device", lambda *a, **kw: None)
    monkeypatch.setattr(rlk, "_run_linear", product)
    refuses(head_linear, tensors("cpu"))
    ways.clear()
    head_linear(**tensors("cpu"))
    assert ways == ["product"]


@pytest.mark.gpu
def test_differentiable_calls_refuse():
    dev = torch.device("cuda")
    t = tensors(dev)
    refuses(head_linear, t)
    targets = torch.zeros(N, dtype=torch.int32, device=dev)
    rules = rlk.LogitRules(temperature=torch.ones(N, device=dev))
    refuses(lambda x: rlk.processed_selected_token_logprob(x, targets, rules, real_vocab=K),
            {"x": t["x"]})
    refuses(lambda x: rlk.selected_token_logprob(x, targets, real_vocab=K), {"x": t["x"]})
    head = torch.ones(256, K, dtype=torch.bfloat16, device=dev)  # (the least that a tile takes)
    refuses(lambda x, weight: rlk.lmhead_selected_token_logprob(x, weight, targets, real_vocab=V,
                                                                num_vocab_tiles=1),
            {"x": t["x"], "weight": head})
