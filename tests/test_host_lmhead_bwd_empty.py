"""The LM-head's gradients of a batch without tokens (no GPU: nothing launches a kernel).  An
empty tensor has no address, so its pointers are NULL."""
from __future__ import annotations

import pytest

import vocab_selected_token_amd as rlk


class NoStream:
    cuda_stream = 0


def call(num_tokens):
    d = rlk.make_desc(num_tokens, 1000, 1024, 1024, 4)
    rlk.rlk_logp_fused_lmhead_bwd(d, None, None, 64, None, None, None, None, None, None, None,
                                  None, stream=NoStream())


def test_only_the_hidden_gradient_of_nothing():
    call(0)


def test_no_output_of_tokens_is_refused():
    with pytest.raises(rlk.RlkError) as ei:
        call(8)
    assert ei.value.status == rlk.RLK_ERR_NULL_POINTER
