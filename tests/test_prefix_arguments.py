"""Arguments of the shared-prefix attention and the preparation that the binding has to refuse, or to take as the other entries do."""
import numpy as np
import pytest
import torch

import exact_long_sequence_gb300 as ela

from test_binding_streams import Tensor, bf16, machine, ready_args  # noqa: F401


def call(**over):
    a = dict(q=bf16(3, 8, 1, 64), k_prefix=bf16(2, 100, 64), v_prefix=bf16(2, 100, 64), k_own=bf16(3, 2, 20, 64),
             v_own=bf16(3, 2, 20, 64), own_lens=Tensor((3,), torch.int32))
    return ela.attn_fwd_prefix(**{**a, **over})


@pytest.mark.parametrize("over", [dict(k_prefix=None), dict(v_prefix=None), dict(k_own=None), dict(v_own=None)], ids=str)
def test_keys_and_values_come_together(machine, over):  # noqa: F811
    """A V without its K is a mistake of the caller, not a call without that part."""
    with pytest.raises(ValueError):
        call(**over)
    assert not machine.lib.calls


def test_each_part_may_be_left_out_whole(machine):  # noqa: F811
    call(k_prefix=None, v_prefix=None)
    call(k_own=None, v_own=None)
    call(k_own=None, v_own=None, own_lens=None)
    assert len(machine.lib.calls) == 3


def test_numbers_of_other_types_are_taken_as_the_other_entries_take_them(machine, monkeypatch):  # noqa: F811
    """scale and eps may be anything float() takes, as attn_fwd's scale and layernorm_rows' eps."""
    for number in (np.float32(0.25), torch.tensor(0.25), np.array(0.25)):
        calls = []
        for name in ("attn_fwd_prefix", "attn_qk_norm_rope", "attn_qk_norm_rope_bwd"):
            monkeypatch.setattr(machine.lib, name, lambda *a: calls.append(a) or ela.ATTN_OK, raising=False)
        call(scale=number)
        ela.qk_norm_rope(*ready_args(), eps=number)
        ela.qk_norm_rope_bwd(bf16(2, 4, 6, 64), bf16(2, 2, 6, 64), *ready_args(), eps=number)
        assert len(calls) == 3
        assert all(any(type(x) is float and x == 0.25 for x in a) for a in calls)
