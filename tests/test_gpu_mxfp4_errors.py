"""Who learns of a product's timed out wait: its own stream's workspace, or all
calls that share one and are checked together."""
import pytest
import torch

from jagged_attention_recommender_jfa_b200 import jfa
from test_gpu_mxfp4 import draw

pytestmark = pytest.mark.gpu


def timed_out(ws, stream):
    with pytest.raises(jfa.JfaError) as ei:
        jfa.jfa_check_error(ws, stream)
    assert ei.value.status == jfa.JFA_ERR_TIMEOUT


@pytest.fixture
def products(cuda_device):
    """Two products (a split contraction, pairs of CTAs), their results and a stream for each."""
    out = []
    for m, n, k in ((64, 64, 8192), (300, 512, 8192)):
        a, b = (jfa.quantize_mxfp4(draw(r, k, "bf16", r).to(cuda_device)) for r in (m, n))
        out.append((a, b, jfa.matmul_mxfp4(a, b), torch.cuda.Stream(cuda_device)))
    torch.cuda.synchronize()
    return out


def run(p, ws, inject=False):
    a, b, _, stream = p
    if inject:
        jfa.jfa_test_inject(jfa.JFA_TEST_MATMUL_SKIP_LOAD)
    return jfa.matmul_mxfp4(a, b, ws=ws, stream=stream, check=False)


@pytest.mark.parametrize("failing", [0, 1])
def test_streams_with_a_workspace_each(cuda_device, products, failing):
    ws = [jfa.mxfp4_workspace(cuda_device) for _ in products]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [run(p, w, i == failing) for i, (p, w) in enumerate(zip(products, ws))]
        timed_out(ws[failing], products[failing][3])
        jfa.jfa_check_error(ws[1 - failing], products[1 - failing][3])
        assert torch.equal(got[1 - failing], products[1 - failing][2])


@pytest.mark.parametrize("failing", [0, 1])
def test_streams_that_share_a_workspace_are_checked_together(cuda_device, products, failing):
    ws = jfa.mxfp4_workspace(cuda_device)
    torch.cuda.synchronize()
    for _ in range(3):
        for i, p in enumerate(products):
            run(p, ws, i == failing)
        torch.cuda.synchronize()
        timed_out(ws, None)
        # read and cleared: the next calls are right and found so
        got = [run(p, ws) for p in products]
        torch.cuda.synchronize()
        jfa.jfa_check_error(ws)
        assert all(torch.equal(g, p[2]) for g, p in zip(got, products))


def test_an_attention_call_leaves_a_product_armed(cuda_device, products):
    # the injected failure reaches the product that it is meant for
    q = torch.randn(64, 1, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(cuda_device)
    off = torch.tensor([0, 64], dtype=torch.int32, device=cuda_device)
    prob = jfa.make_problem(batch=1, heads=1, head_dim=128, max_q_len=64, max_kv_len=64, total_q=64, total_kv=64,
                            dtype="bf16")
    assert jfa.jfa_path(prob, "softmax", 0) == 1
    want = jfa.attention_forward(prob, q, q, q, off, off)[0]
    ws = jfa.mxfp4_workspace(cuda_device)
    torch.cuda.synchronize()
    jfa.jfa_test_inject(jfa.JFA_TEST_MATMUL_SKIP_LOAD)
    assert torch.equal(jfa.attention_forward(prob, q, q, q, off, off)[0], want)
    run(products[0], ws)
    timed_out(ws, products[0][3])
    got = run(products[0], ws)
    jfa.jfa_check_error(ws, products[0][3])
    assert torch.equal(got, products[0][2])
