"""Refusals of the binding of the operators around the two blocks that need no GPU."""
import pytest
import torch

import long_context_attention_upipe_gb300 as up


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_attention_upipe_gb300 import _build
    _build.build()


@pytest.mark.parametrize("k,q_out,k_out", [(True, True, False), (True, False, True), (True, False, False), (False, False, False)])
def test_rope_refuses_a_missing_output(k, q_out, k_out):
    x = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 4, dtype=torch.int32)
    n = up.launch_count()
    with pytest.raises(ValueError, match="output"):
        up.rope(up.make_rope_desc(64, [0.5] * 32), x, x if k else None, pos, x if q_out else None, x if k_out else None)
    assert up.launch_count() == n
