"""One tensor as several of a call's rules: each is checked as what it is passed as (no GPU)."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk

AT = torch.zeros(4, dtype=torch.int64)


@pytest.mark.parametrize("name, table", [("bias", torch.zeros(2, 100)),
                                         ("allow", torch.zeros(2, 4, dtype=torch.int32))])
def test_a_history_that_is_an_index_too_needs_an_element_per_row(name, table):
    """Row r's index is read at [r]: one of fewer elements than rows would be read past its end."""
    for tokens in (0, 3, 5):
        h = torch.zeros(tokens, dtype=torch.int32)
        with pytest.raises(ValueError, match=f"{name}_index has {tokens} elements, other rules 4"):
            rlk.LogitRules(history=h, history_begin=AT, history_end=AT,
                           **{name: table, name + "_index": h})
    h = torch.zeros(4, dtype=torch.int32)
    assert rlk.LogitRules(history=h, history_begin=AT, history_end=AT,
                          **{name: table, name + "_index": h}).rows == 4


def test_one_index_for_both_tables():
    i = torch.zeros(4, dtype=torch.int32)
    r = rlk.LogitRules(bias=torch.zeros(2, 100), bias_index=i,
                       allow=torch.zeros(2, 4, dtype=torch.int32), allow_index=i)
    assert r.rows == 4 and r.struct.bias_index == r.struct.allow_index == i.data_ptr()
