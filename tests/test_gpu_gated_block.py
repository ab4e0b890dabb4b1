"""The operators around the attention, run together as a block of the model
uses them: pre norm -> MXFP4 projections -> jagged attention -> norm, gate and
residual scale -> the next block's projection, forward and backward, with the
jagged batch's offsets.

Every stage is compared with its 64-bit form on the values the stage was
given (a quantiser's code is an integer decision, so an end-to-end comparison
would compare flipped codes, not errors): norms and products with the bounds
of their own tests, the attention with the framework's parity bounds.  The
same block captured in a graph and replayed on other data gives the bits of
the eager run.
"""
import numpy as np
import pytest
import torch

import oracle
from jagged_attention_recommender_jfa_b200 import jfa
from oracle import mx4

pytestmark = pytest.mark.gpu

H, HD = 2, 128
D = H * HD
EPS = 1e-5


class Block:
    """Weights of one gated attention block (projections to q, k, v and the gate u)."""

    def __init__(self, dev, seed):
        g = torch.Generator().manual_seed(seed)
        w = torch.randn(4 * D, D, generator=g) / D ** 0.5
        self.w = w.to(torch.bfloat16).to(dev)
        self.w_next = (torch.randn(3 * HD, D, generator=g) / D ** 0.5).to(torch.bfloat16).to(dev)
        vec = lambda c: (c + 0.2 * torch.randn(D, generator=g)).to(dev)
        self.scale, self.post_gamma, self.pre_gamma, self.first_gamma = vec(0.5), vec(1), vec(1), vec(1)
        self.table = (0.3 * torch.randn(H, 2 * 300 + 1, generator=g)).to(dev)
        # once per training step
        self.op, self.op_t = jfa.quantize_mxfp4(self.w), jfa.quantize_mxfp4(self.w, along_rows=True)
        self.next_op, self.next_t = jfa.quantize_mxfp4(self.w_next), jfa.quantize_mxfp4(self.w_next, along_rows=True)


class Batch:
    def __init__(self, dev, lens, seed):
        self.lens = lens
        self.rows = sum(lens)
        off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.off = torch.from_numpy(off).to(dev)
        g = torch.Generator().manual_seed(seed)
        t = lambda c: torch.randn(self.rows, c, generator=g).to(torch.bfloat16).to(dev)
        self.x, self.before, self.dz, self.dy = t(D), t(D), t(3 * HD), t(D)
        self.prob = jfa.make_problem(batch=len(lens), heads=H, head_dim=HD, max_q_len=300, max_kv_len=300,
                                     total_q=self.rows, total_kv=self.rows, dtype="bf16", bias_kind="relpos",
                                     relpos_len=601)
        self.first = jfa.make_block_norm(rows=self.rows, dim=D, post_norm="none", pre_norm="rms", gate="none", eps=EPS)
        self.desc = jfa.make_block_norm(rows=self.rows, dim=D, eps=EPS)


def forward(b, t, ws, aws):
    """Residual stream in and out; every intermediate value."""
    r = {}
    r["x"], r["n"] = jfa.block_norm_forward(t.first, t.x, t.before, pre_gamma=b.first_gamma)
    r["qkvu"] = jfa.linear_mxfp4_forward(r["n"], b.op, ws=ws, check=False)
    r["q"], r["k"], r["v"], r["u"] = (p.contiguous() for p in r["qkvu"].chunk(4, dim=1))
    heads = lambda z: z.view(t.rows, H, HD)
    r["o"], r["lse"] = jfa.attention_forward(t.prob, heads(r["q"]), heads(r["k"]), heads(r["v"]), t.off, t.off, b.table,
                                             "softmax", True, ws=aws, check=False)
    r["y"], r["m"] = jfa.block_norm_forward(t.desc, r["x"], r["o"].view(t.rows, D), r["u"], b.scale, b.post_gamma,
                                            pre_gamma=b.pre_gamma)
    r["z"] = jfa.linear_mxfp4_forward(r["m"], b.next_op, ws=ws, check=False)
    return r


def backward(b, t, r, ws, aws, nws):
    """Gradients of <dz, z> + <dy, y>."""
    g = {}
    g["m"], g["w_next"] = jfa.linear_mxfp4_backward(t.dz, r["m"], b.next_t, ws=ws, check=False)
    n = jfa.block_norm_backward(t.desc, r["x"], r["o"].view(t.rows, D), r["u"], b.scale, b.post_gamma,
                                pre_gamma=b.pre_gamma, dy=t.dy, dn=g["m"], ws=nws)
    g["norm"] = n
    heads = lambda z: z.view(t.rows, H, HD)
    dq, dk, dv, g["table"] = jfa.attention_backward(
        t.prob, heads(r["q"]), heads(r["k"]), heads(r["v"]), r["o"], r["lse"], heads(n["block"]), t.off, t.off, b.table,
        "softmax", True, ws=aws, check=False, want_dbias=True)
    g["qkvu"] = torch.cat([z.reshape(t.rows, D) for z in (dq, dk, dv)] + [n["gate"]], dim=1)
    g["n"], g["w"] = jfa.linear_mxfp4_backward(g["qkvu"], r["n"], b.op_t, ws=ws, check=False)
    g["first"] = jfa.block_norm_backward(t.first, t.x, t.before, pre_gamma=b.first_gamma, dy=n["x"], dn=g["n"])
    return g


def workspaces(t, dev):
    return (jfa.mxfp4_workspace(dev), jfa.workspace(t.prob, False, dev), jfa.workspace(t.prob, True, dev),
            jfa.block_norm_workspace(t.desc, dev))


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, ref, bound, what):
    g = f64(got)
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    bad = ~(np.abs(g - ref) <= bound)
    assert g.shape == ref.shape and not bad.any(), (what, np.argwhere(bad)[:3])


def check_product(got, a, b, what):
    """got against the product of the quantised rows of a and of b."""
    A, B = (mx4.values(*mx4.quantize(t), t.shape[1]) for t in (a, b))
    near(got, A @ B.T, (a.shape[1] + 24) * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T), what)


def check_norm(got, ref, what, chain=340):
    near(got, ref[0], chain * 2.0 ** -24 * ref[1], what)


@pytest.mark.parametrize("lens", [[1], [5, 0, 130, 17], [300, 64, 65, 1, 128]])
def test_block_forward_and_backward(cuda_device, lens):
    dev = cuda_device
    b, t = Block(dev, 1), Batch(dev, lens, 2)
    ws, aws, bws, nws = workspaces(t, dev)
    r = forward(b, t, ws, aws)
    jfa.jfa_check_error(aws)
    g = backward(b, t, r, ws, bws, nws)
    jfa.jfa_check_error(bws)
    jfa.jfa_check_error(ws)
    # forward, stage by stage
    eps = np.float32(EPS)
    first = dict(post="none", pre="rms", gate_kind="none", eps=eps, pre_gamma=f64(b.first_gamma))
    ref = mx4.block_norm(f64(t.x), f64(t.before), **first)
    check_norm(r["x"], ref["y"], "x")
    check_norm(r["n"], ref["n"], "n")
    check_product(r["qkvu"], f64(r["n"]), f64(b.w), "qkvu")
    kw = dict(bias=b.table.cpu(), bias_kind="relpos", relpos_len=601, act="softmax", causal=True)
    off = t.off.cpu().numpy()
    heads = lambda z: f64(z).reshape(t.rows, H, HD)
    ro, _ = oracle.forward(off, off, heads(r["q"]), heads(r["k"]), heads(r["v"]), **kw)
    near(r["o"], ro, np.full(ro.shape, 2e-2), "o")
    mid = dict(gate=f64(r["u"]), scale=f64(b.scale), post_gamma=f64(b.post_gamma), pre_gamma=f64(b.pre_gamma), eps=eps)
    o = f64(r["o"]).reshape(t.rows, D)
    ref = mx4.block_norm(f64(r["x"]), o, **mid)
    check_norm(r["y"], ref["y"], "y")
    check_norm(r["m"], ref["n"], "m")
    check_product(r["z"], f64(r["m"]), f64(b.w_next), "z")
    # backward, stage by stage
    check_product(g["m"], f64(t.dz), f64(b.w_next).T, "dm")
    check_product(g["w_next"], f64(t.dz).T, f64(r["m"]).T, "dw_next")
    ref = mx4.block_norm(f64(r["x"]), o, **mid, dy=f64(t.dy), dn=f64(g["m"]))
    for name in ("x", "block", "gate"):
        check_norm(g["norm"][name], ref[name], name)
    for name in ("scale", "post_gamma", "pre_gamma"):
        check_norm(g["norm"][name], ref[name], name, 540)
    rdq, rdk, rdv = oracle.backward(off, off, heads(r["q"]), heads(r["k"]), heads(r["v"]), heads(g["norm"]["block"]), **kw)
    for i, rd in enumerate((rdq, rdk, rdv)):
        near(g["qkvu"][:, i * D:(i + 1) * D], rd.reshape(t.rows, D), np.full((t.rows, D), 2e-2), "dqkv"[:1] + "qkv"[i])
    assert torch.equal(g["qkvu"][:, 3 * D:], g["norm"]["gate"])
    check_product(g["n"], f64(g["qkvu"]), f64(b.w).T, "dn")
    check_product(g["w"], f64(g["qkvu"]).T, f64(r["n"]).T, "dw")
    ref = mx4.block_norm(f64(t.x), f64(t.before), **first, dy=f64(g["norm"]["x"]), dn=f64(g["n"]))
    check_norm(g["first"]["x"], ref["x"], "dx")
    check_norm(g["first"]["block"], ref["block"], "dbefore")
    check_norm(g["first"]["pre_gamma"], ref["pre_gamma"], "dgamma", 540)


def test_block_in_a_graph(cuda_device):
    dev = cuda_device
    b = Block(dev, 3)
    lens = [33, 200, 0, 71]
    batches = [Batch(dev, lens, s) for s in (4, 5)]
    t = Batch(dev, lens, 6)
    ws, aws, bws, nws = workspaces(t, dev)
    step = lambda z: (lambda r: (r, backward(b, z, r, ws, bws, nws)))(forward(b, z, ws, aws))
    step(t)   # loads modules before the capture
    want = [step(z) for z in batches]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, g = step(t)
    for z, (wr, wg) in zip(batches, want):
        for name in ("x", "before", "dz", "dy"):
            getattr(t, name).copy_(getattr(z, name))
        graph.replay()
        torch.cuda.synchronize()
        for name in ("z", "y", "qkvu"):
            assert torch.equal(r[name], wr[name]), name
        # past the attention's backward (its sums over query tiles have no
        # fixed order) values agree to its rounding, before it in every bit
        for name in ("m", "w_next"):
            assert torch.equal(g[name], wg[name]), name
        for name in ("x", "block", "gate", "scale", "post_gamma", "pre_gamma"):
            assert torch.equal(g["norm"][name], wg["norm"][name]), name
    jfa.jfa_check_error(ws)


def test_streams_side_by_side(cuda_device):
    # products (their kernels take whole SMs and all of their tensor memory),
    # norms and the attention on three streams at once, a stream given by its
    # handle among them
    dev = cuda_device
    b, t = Block(dev, 7), Batch(dev, [300] * 12, 8)
    ws, aws, _, nws = workspaces(t, dev)
    r = forward(b, t, ws, aws)
    big = jfa.quantize_mxfp4(torch.randn(6000, 1024, generator=torch.Generator().manual_seed(1)).to(dev))
    w = jfa.quantize_mxfp4(torch.randn(2048, 1024, generator=torch.Generator().manual_seed(2)).to(dev))
    heads = lambda z: z.view(t.rows, H, HD)
    attend = lambda **kw: jfa.attention_forward(t.prob, heads(r["q"]), heads(r["k"]), heads(r["v"]), t.off, t.off, b.table,
                                                "softmax", True, ws=aws, check=False, **kw)[0]
    norm = lambda **kw: jfa.block_norm_backward(t.desc, r["x"], r["o"].view(t.rows, D), r["u"], b.scale, b.post_gamma,
                                                pre_gamma=b.pre_gamma, dy=t.dy, dn=t.dy, ws=nws, **kw)
    product = lambda **kw: jfa.matmul_mxfp4(big, w, ws=ws, check=False, **kw)
    want = product(), norm(), attend()
    streams = [torch.cuda.Stream(dev) for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append((product(stream=streams[0]), norm(stream=streams[1].cuda_stream), attend(stream=streams[2])))
    torch.cuda.synchronize()
    for p, n, o in got:
        assert torch.equal(p, want[0]) and torch.equal(o, want[2])
        assert all(torch.equal(n[k], want[1][k]) for k in n if n[k] is not None)
    assert torch.equal(jfa.matmul_mxfp4(big, w, ws=ws, stream=0), want[0])
    jfa.jfa_check_error(aws)
