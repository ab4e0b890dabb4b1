"""Host-side checks of the operators around the attention (no GPU needed):
buffer sizes, and that bad arguments are refused before anything is enqueued."""
import pytest
import torch

from jagged_attention_recommender_jfa_b200 import jfa
from oracle import mx4

FAKE = 1 << 20   # never dereferenced: every case fails host validation or is empty
INVALID, UNSUPPORTED, WORKSPACE = (jfa.JFA_ERR_INVALID_ARGUMENT, jfa.JFA_ERR_UNSUPPORTED,
                                   jfa.JFA_ERR_WORKSPACE)


def refused(status, fn, *a, **kw):
    with pytest.raises(jfa.JfaError) as ei:
        fn(*a, **kw)
    assert ei.value.status == status, str(ei.value)


@pytest.mark.parametrize("rows,cols", [(0, 0), (1, 1), (1, 32), (127, 33), (129, 128), (1000, 1003), (5, 4097)])
def test_operand_sizes(rows, cols):
    blocks = mx4.ceil_div(cols, 32)
    assert jfa.jfa_mxfp4_code_bytes(rows, cols) == rows * blocks * 16
    assert jfa.jfa_mxfp4_scale_bytes(rows, cols) == mx4.scale_bytes(rows, blocks)


def test_operand_sizes_out_of_range():
    big = (1 << 30) + 1
    for r, c in ((-1, 32), (1, -1), (big, 1), (1, big)):
        assert jfa.jfa_mxfp4_code_bytes(r, c) == 0 and jfa.jfa_mxfp4_scale_bytes(r, c) == 0
    assert jfa.jfa_mxfp4_code_bytes(1 << 30, 1 << 20) == 1 << 49


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), INVALID), (dict(dtype=7), INVALID), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID),
    (dict(rows=(1 << 30) + 1), INVALID), (dict(cols=(1 << 30) + 1), INVALID), (dict(x=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(codes=FAKE + 4), INVALID), (dict(scales=FAKE + 1), INVALID)])
@pytest.mark.parametrize("dequant", [False, True])
def test_quantiser_refusals(change, status, dequant):
    a = dict(x=FAKE, dtype="bf16", rows=10, cols=64, along_rows=0, codes=FAKE, scales=FAKE)
    a.update(change)
    if dequant:
        refused(status, jfa.jfa_quantize_mxfp4_dequant, **a, dequant=FAKE, stream=0)
    else:
        refused(status, jfa.jfa_quantize_mxfp4, **a, stream=0)


@pytest.mark.parametrize("change", [dict(dtype=2), dict(rows=-1), dict(cols=(1 << 30) + 1), dict(x=None), dict(codes=None),
                                    dict(scales_t=None), dict(codes_t=None), dict(codes_t=FAKE + 8), dict(x=FAKE + 2)])
def test_two_way_quantiser_refusals(change):
    a = dict(x=FAKE, dtype="bf16", rows=10, cols=64, codes=FAKE, scales=FAKE, codes_t=FAKE, scales_t=FAKE)
    refused(INVALID, jfa.jfa_quantize_mxfp4_both, **{**a, **change}, stream=0)


def test_quantiser_dequant_pointer_and_empty():
    refused(INVALID, jfa.jfa_quantize_mxfp4_dequant, FAKE, "f32", 3, 3, 0, FAKE, FAKE, None, stream=0)
    refused(INVALID, jfa.jfa_quantize_mxfp4_dequant, FAKE, "f32", 3, 3, 1, FAKE, FAKE, FAKE + 4, stream=0)
    jfa.jfa_quantize_mxfp4(None, "bf16", 0, 64, 0, None, None, stream=0)
    jfa.jfa_quantize_mxfp4(None, "bf16", 64, 0, 1, None, None, stream=0)
    jfa.jfa_quantize_mxfp4_both(None, "bf16", 0, 64, None, None, None, None, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(k=-1), INVALID), (dict(m=(1 << 30) + 1), INVALID),
    (dict(out_dtype=2), INVALID), (dict(a_codes=None), INVALID), (dict(a_scales=None), INVALID),
    (dict(b_codes=None), INVALID), (dict(b_scales=None), INVALID), (dict(out=None), INVALID),
    (dict(workspace=None), INVALID), (dict(ws_bytes=255), WORKSPACE), (dict(a_codes=FAKE + 8), INVALID),
    (dict(b_scales=FAKE + 4), INVALID), (dict(out=FAKE + 8), INVALID), (dict(bias=FAKE + 2), INVALID),
    (dict(workspace=FAKE + 8), INVALID)])
def test_product_refusals(change, status):
    a = dict(m=4, n=8, k=32, a_codes=FAKE, a_scales=FAKE, b_codes=FAKE, b_scales=FAKE, bias=None, out=FAKE,
             out_dtype="f32", accumulate=0, workspace=FAKE, ws_bytes=256)
    a.update(change)
    refused(status, jfa.jfa_matmul_mxfp4, **a, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(n=(1 << 30) + 1), INVALID), (dict(k=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID), (dict(w_codes=None), INVALID), (dict(w_scales=None), INVALID),
    (dict(w_codes=FAKE + 4), INVALID), (dict(y=None), INVALID), (dict(y=FAKE + 2), INVALID), (dict(bias=FAKE + 2), INVALID),
    (dict(scratch=None), INVALID), (dict(scratch=FAKE + 8), INVALID), (dict(scratch_bytes=575), WORKSPACE),
    (dict(workspace=None), INVALID), (dict(workspace=FAKE + 8), INVALID), (dict(ws_bytes=255), WORKSPACE)])
def test_linear_forward_refusals(change, status):
    assert jfa.jfa_linear_mxfp4_scratch_bytes(4, 8, 32, 0) == 4 * 16 + 512
    a = dict(x=FAKE, dtype="bf16", m=4, n=8, k=32, w_codes=FAKE, w_scales=FAKE, bias=None, y=FAKE, scratch=FAKE,
             scratch_bytes=576, workspace=FAKE, ws_bytes=256)
    refused(status, jfa.jfa_linear_mxfp4_forward, **{**a, **change}, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(m=(1 << 30) + 1), INVALID), (dict(n=-1), INVALID), (dict(k=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(x_dtype=3), INVALID), (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(wt_codes=None), INVALID), (dict(wt_scales=FAKE + 1), INVALID), (dict(dx=None), INVALID),
    (dict(dw=None), INVALID), (dict(dw=FAKE + 4), INVALID), (dict(scratch=None), INVALID),
    (dict(scratch_bytes=2239), WORKSPACE), (dict(workspace=None), INVALID), (dict(ws_bytes=0), WORKSPACE)])
def test_linear_backward_refusals(change, status):
    # dy 4 x 8, its transpose and x's (32 x 4)
    assert jfa.jfa_linear_mxfp4_scratch_bytes(4, 8, 32, 1) == (4 + 8 + 32) * 16 + 3 * 512 == 2240
    a = dict(dy=FAKE, dtype="bf16", x=FAKE, x_dtype="f32", m=4, n=8, k=32, wt_codes=FAKE, wt_scales=FAKE, dx=FAKE, dw=FAKE,
             accumulate=0, scratch=FAKE, scratch_bytes=2240, workspace=FAKE, ws_bytes=256)
    refused(status, jfa.jfa_linear_mxfp4_backward, **{**a, **change}, stream=0)


def test_linear_of_nothing_is_a_no_op():
    assert jfa.jfa_linear_mxfp4_scratch_bytes(-1, 8, 8, 0) == jfa.jfa_linear_mxfp4_scratch_bytes(8, 8, (1 << 30) + 1, 1) == 0
    jfa.jfa_linear_mxfp4_forward(None, "bf16", 0, 8, 32, None, None, None, None, None, FAKE, 0, 256, stream=0)
    jfa.jfa_linear_mxfp4_forward(FAKE, "bf16", 3, 0, 32, None, None, None, None, FAKE, FAKE, 1 << 20, 256, stream=0)
    jfa.jfa_linear_mxfp4_backward(FAKE, "f32", None, "f32", 3, 8, 0, None, None, None, None, 0, FAKE, FAKE, 1 << 20, 256,
                                  stream=0)


def test_product_of_nothing_is_a_no_op():
    assert jfa.jfa_mxfp4_workspace_bytes() == 256
    for m, n in ((0, 8), (8, 0)):
        jfa.jfa_matmul_mxfp4(m, n, 32, None, None, None, None, None, None, "bf16", 0, FAKE, 256, stream=0)


def _norm_args(**change):
    a = dict(x=FAKE, block=FAKE, gate=FAKE, scale=FAKE, post_gamma=FAKE, post_beta=None, pre_gamma=FAKE,
             pre_beta=None)
    a.update(change)
    return a


DESC = [(dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(dim=0), INVALID), (dict(dim=8193), UNSUPPORTED),
        (dict(dtype=2), INVALID), (dict(post_norm=3), INVALID), (dict(pre_norm=-1), INVALID), (dict(gate=4), INVALID),
        (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
        (dict(eps=float("inf")), INVALID)]


@pytest.mark.parametrize("change,status", DESC)
def test_block_norm_descriptor_refusals(change, status):
    d = jfa.make_block_norm(**{**dict(rows=4, dim=64), **change})
    assert jfa.jfa_block_norm_workspace_bytes(d) == 0
    refused(status, jfa.jfa_block_norm_forward, d, **_norm_args(), y=FAKE, n=FAKE, stream=0)
    refused(status, jfa.jfa_block_norm_backward, d, **_norm_args(), dy=FAKE, dn=FAKE, dx=FAKE, dblock=FAKE,
            dgate=FAKE, dscale=FAKE, dpost_gamma=FAKE, dpost_beta=None, dpre_gamma=FAKE, dpre_beta=None,
            workspace=FAKE, ws_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("kinds,change", [
    ({}, dict(x=None)), ({}, dict(block=None)), ({}, dict(gate=None)), ({}, dict(x=FAKE + 8)),
    ({}, dict(gate=FAKE + 2)), ({}, dict(scale=FAKE + 4)), ({}, dict(post_beta=FAKE)), ({}, dict(pre_beta=FAKE)),
    (dict(post_norm="none"), {}), (dict(pre_norm="none"), {}), (dict(gate="none"), {})])
def test_block_norm_argument_refusals(kinds, change):
    d = jfa.make_block_norm(rows=4, dim=64, **kinds)
    refused(INVALID, jfa.jfa_block_norm_forward, d, **_norm_args(**change), y=FAKE, n=FAKE, stream=0)
    refused(INVALID, jfa.jfa_block_norm_backward, d, **_norm_args(**change), dy=FAKE, dn=FAKE, dx=FAKE, dblock=FAKE,
            dgate=FAKE, dscale=FAKE, dpost_gamma=FAKE, dpost_beta=None, dpre_gamma=FAKE, dpre_beta=None,
            workspace=FAKE, ws_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(y=None), INVALID), (dict(n=None), INVALID), (dict(y=FAKE + 8), INVALID)])
def test_block_norm_forward_result_refusals(change, status):
    d = jfa.make_block_norm(rows=4, dim=64)
    refused(status, jfa.jfa_block_norm_forward, d, **_norm_args(), **{**dict(y=FAKE, n=FAKE), **change}, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), INVALID), (dict(dn=None), INVALID), (dict(dx=None), INVALID), (dict(dblock=None), INVALID),
    (dict(dgate=None), INVALID), (dict(dx=FAKE + 4), INVALID), (dict(dpost_beta=FAKE), INVALID),
    (dict(dscale=FAKE + 4), INVALID), (dict(workspace=None), INVALID), (dict(workspace=FAKE + 4), INVALID),
    (dict(ws_bytes=16), WORKSPACE)])
def test_block_norm_backward_result_refusals(change, status):
    d = jfa.make_block_norm(rows=4, dim=64)
    a = dict(dy=FAKE, dn=FAKE, dx=FAKE, dblock=FAKE, dgate=FAKE, dscale=FAKE, dpost_gamma=FAKE, dpost_beta=None,
             dpre_gamma=FAKE, dpre_beta=None, workspace=FAKE, ws_bytes=jfa.jfa_block_norm_workspace_bytes(d))
    a.update(change)
    refused(status, jfa.jfa_block_norm_backward, d, **_norm_args(), **a, stream=0)


def test_block_norm_forward_of_no_rows_is_a_no_op():
    d = jfa.make_block_norm(rows=0, dim=64)
    jfa.jfa_block_norm_forward(d, None, None, None, None, None, None, None, None, None, None, stream=0)
    assert jfa.jfa_block_norm_workspace_bytes(d) > 0


def test_conveniences_refuse_host_and_misshapen_tensors():
    x = torch.zeros(4, 64)
    refused(INVALID, jfa.quantize_mxfp4, x)                       # not on a GPU
    refused(INVALID, jfa.quantize_mxfp4, torch.zeros(4, 4, 4))
    refused(INVALID, jfa.quantize_mxfp4, torch.zeros(4, 64, dtype=torch.float16))
    op = jfa.MxOperand(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64)
    refused(INVALID, jfa.matmul_mxfp4, op, op)
    refused(INVALID, jfa.matmul_mxfp4, x, op)
    refused(INVALID, jfa.matmul_mxfp4, op._replace(rows=5), op)
    d = jfa.make_block_norm(rows=4, dim=64, dtype="f32")
    refused(INVALID, jfa.block_norm_forward, d, x, x, x)
    refused(INVALID, jfa.linear_mxfp4_backward, x, torch.zeros(5, 64), op)
