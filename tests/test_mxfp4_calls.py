"""Host-side checks of the workspaces of the operators around the attention
(no GPU needed)."""
import pytest
import torch

from jagged_attention_recommender_jfa_b200 import jfa


def refused(match, fn, *a, **kw):
    with pytest.raises(jfa.JfaError, match=match) as ei:
        fn(*a, **kw)
    assert ei.value.status == jfa.JFA_ERR_INVALID_ARGUMENT


def test_an_error_word_that_nobody_could_read_is_refused():
    op = jfa.MxOperand(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64)
    x = torch.zeros(4, 64)
    refused("needs ws", jfa.matmul_mxfp4, op, op, check=False)
    refused("needs ws", jfa.linear_mxfp4_forward, x, op, check=False)
    refused("needs ws", jfa.linear_mxfp4_backward, x, x, op, check=False)
    # with a workspace the calls go on to their other arguments
    ws = torch.zeros(256, dtype=torch.uint8)
    refused("device cpu", jfa.matmul_mxfp4, op, op, ws=ws, check=False)
    refused("device cpu", jfa.linear_mxfp4_forward, x, op, ws=ws, check=False)
    refused("device cpu", jfa.linear_mxfp4_backward, x, x, op, ws=ws, check=False)
