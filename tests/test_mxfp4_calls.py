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


# 256 bytes by their element count, one or 511 in memory
STRIDED = [torch.zeros(1, dtype=torch.uint8).expand(256), torch.zeros(512, dtype=torch.uint8)[::2]]
FAKE = 1 << 20   # never dereferenced


@pytest.mark.parametrize("ws", STRIDED)
def test_workspaces_without_their_memory_are_refused(ws):
    assert ws.numel() * ws.element_size() == jfa.jfa_mxfp4_workspace_bytes()
    refused("contiguous", jfa._ws_on, ws, -1)
    refused("contiguous", jfa._ws_on, "ws", -1)
    refused("contiguous", jfa.jfa_matmul_mxfp4, 4, 8, 32, FAKE, FAKE, FAKE, FAKE, None, FAKE, "bf16", 0, ws)
    refused("contiguous", jfa.jfa_linear_mxfp4_forward, FAKE, "bf16", 4, 8, 32, FAKE, FAKE, None, FAKE, ws, FAKE,
            ws_bytes=256)
    d = jfa.make_block_norm(rows=1, dim=1, post_norm="none", pre_norm="none", gate="none")
    refused("contiguous", jfa.jfa_block_norm_backward, d, FAKE, FAKE, None, None, None, None, None, None, FAKE, None,
            FAKE, FAKE, None, None, None, None, None, None, ws)
    ok = torch.zeros(256, dtype=torch.uint8)
    assert jfa._ws_on(ok, -1) is ok and jfa._nbytes(ok) == 256 == jfa._nbytes(FAKE, 256)
