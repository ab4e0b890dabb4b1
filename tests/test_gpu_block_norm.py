"""The norms before and after a block on the GPU, forward and backward,
against the 64-bit forms (oracle.mx4.block_norm).

Tolerance.  oracle.mx4.block_norm returns a magnitude with each result: an
fp32 evaluation (rounding unit 2^-24) whose longest chain of operations is L
stays within L 2^-24 magnitude.  The chain of a row's result: a sum over up
to 8192 elements is 16 additions in a thread, 5 shuffles and up to 32 warps,
two of those in a row per norm (mean, variance), two norms and one sum on the
way back: 5 x 53 + about 60 elementwise operations (the exponential and the
fast reciprocal count 4 each) < 340.  (Rows of an odd width above 8176 bf16 or
4096 fp32 columns put up to 24 elements in a thread, but then at most 16 warps
and four sums in a row: less.)  Summed over rows: a CTA's rows one
after the other, then partial rows in strands of eight: at most rows / grid +
grid / 8 + 8 < 200 more for these sizes.  A bf16 result adds half a step, 2^-8
of the value.
"""
import itertools

import numpy as np
import pytest
import torch

from jagged_attention_recommender_jfa_b200 import jfa
from oracle import mx4

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
PARAMS = ("scale", "post_gamma", "post_beta", "pre_gamma", "pre_beta")


def make(rows, dim, dtype, post, pre, gate, seed=0, params=True):
    rng = np.random.default_rng(seed)
    t = lambda mu=0.0: torch.from_numpy(rng.normal(size=(rows, dim)) * np.exp2(rng.integers(-3, 4, (rows, 1))) + mu).to(TORCH[dtype])
    v = lambda c: torch.from_numpy((c + 0.3 * rng.normal(size=dim)).astype(np.float32))
    kw = dict(x=t(), block=t(0.5), gate=t() if gate != "none" else None)
    kw.update(scale=v(0.5) if params else None,
              post_gamma=v(1) if params and post != "none" else None,
              post_beta=v(0) if params and post == "layer" else None,
              pre_gamma=v(1) if params and pre != "none" else None,
              pre_beta=v(0) if params and pre == "layer" else None)
    for name in ("x", "block"):   # padding tokens
        kw[name][rng.random(rows) < 0.1] = 0.0
    return kw, dict(dy=t(), dn=t() if pre != "none" else None)


def dev_(kw, dev):
    return {k: None if t is None else t.to(dev) for k, t in kw.items()}


def np_(kw):
    return {k: None if t is None else t.double().numpy() for k, t in kw.items()}


def close(got, ref, chain, what):
    v, mag = ref
    bound = chain * 2.0 ** -24 * mag
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(v) + bound)
    g = got.double().cpu().numpy()
    assert g.shape == v.shape
    bad = ~(np.abs(g - v) <= bound)
    assert not bad.any(), (what, np.argwhere(bad)[:3], g[bad][:3], v[bad][:3], bound[bad][:3])


def check(dev, rows, dim, dtype, post, pre, gate, seed=0, params=True, eps=1e-5):
    kw, up = make(rows, dim, dtype, post, pre, gate, seed, params)
    desc = jfa.make_block_norm(rows=rows, dim=dim, dtype=dtype, post_norm=post, pre_norm=pre, gate=gate, eps=eps)
    y, n = jfa.block_norm_forward(desc, **dev_(kw, dev))
    g = jfa.block_norm_backward(desc, **dev_(kw, dev), **dev_(up, dev))
    ref = mx4.block_norm(**np_(kw), **np_(up), post=post, pre=pre, gate_kind=gate, eps=np.float32(eps))
    close(y, ref["y"], 340, "y")
    assert (n is None) == (pre == "none")
    if n is not None:
        close(n, ref["n"], 340, "n")
    assert set(g) == set(kw)
    for name, t in kw.items():
        assert (g[name] is None) == (t is None)
        if t is not None:
            close(g[name], ref[name], 540 if name in PARAMS else 340, name)


@pytest.mark.parametrize("post,pre,gate", list(itertools.product(("none", "rms", "layer"), ("none", "rms", "layer"),
                                                            ("none", "identity", "silu", "sigmoid"))))
@pytest.mark.parametrize("dtype,dim", [("f32", 96), ("bf16", 77)])
def test_every_kind(cuda_device, post, pre, gate, dtype, dim):
    check(cuda_device, 37, dim, dtype, post, pre, gate, seed=dim)


@pytest.mark.parametrize("rows,dim", [(1, 1), (5, 2), (1, 7), (3, 8), (9, 33), (130, 64), (257, 255), (50, 256), (21, 257),
                                      (33, 512), (1, 1024), (700, 1024), (40, 1003), (13, 1032), (11, 2050), (6, 4096),
                                      (5, 4097), (7, 4104), (3, 8191), (4, 8192)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_sizes(cuda_device, rows, dim, dtype, kind):
    check(cuda_device, rows, dim, dtype, kind, kind, "silu", seed=rows + dim)


# every count of vectors per thread and both register budgets of wide rows, with
# rows that go round and, in the odd widths, start off the boundaries
@pytest.mark.parametrize("rows,dim", [(310, 4500), (3, 5003), (2, 6144), (310, 6731), (4, 6152), (301, 8185)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", "silu"), ("layer", "layer", "sigmoid"), ("none", "layer", "none")])
def test_wide_rows(cuda_device, rows, dim, dtype, post, pre, gate):
    check(cuda_device, rows, dim, dtype, post, pre, gate, seed=dim)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_parameters(cuda_device, dtype):
    check(cuda_device, 65, 200, dtype, "layer", "rms", "sigmoid", params=False)
    check(cuda_device, 65, 333, dtype, "rms", "layer", "identity", params=False)


def test_many_rows(cuda_device):
    # more rows than the backward has CTAs, small and wide rows
    check(cuda_device, 20001, 40, "bf16", "rms", "rms", "silu")
    check(cuda_device, 3001, 520, "f32", "layer", "layer", "silu")


def test_extreme_gates_stay_finite(cuda_device):
    dim = 64
    u = torch.tensor([-1e4, -200.0, -90.0, -88.5, 0.0, 90.0, 200.0, 1e4] * 8, device=cuda_device).expand(3, dim).contiguous()
    x = torch.randn(3, dim, device=cuda_device)
    for gate in ("silu", "sigmoid"):
        desc = jfa.make_block_norm(rows=3, dim=dim, dtype="f32", post_norm="none", pre_norm="none", gate=gate)
        y, _ = jfa.block_norm_forward(desc, x, x, u)
        g = jfa.block_norm_backward(desc, x, x, u, dy=x)
        s = torch.sigmoid(u.double())
        a = u.double() * s if gate == "silu" else s
        assert torch.allclose(y.double(), x.double() * (1 + a), rtol=2.0 ** -20, atol=1e-30)
        da = s * (1 + u.double() * (1 - s)) if gate == "silu" else s * (1 - s)
        # 1 - s in fp32 is off by the unit of s, times u where that multiplies
        # it; sigmoids below 2^-126 (subnormals) may come out as 0
        assert ((g["gate"].double() - x.double() ** 2 * da).abs()
                <= x.double() ** 2 * (1 + u.double().abs()) * (2.0 ** -20 * s + 2.0 ** -126)).all()


def test_zero_rows_and_constant_rows(cuda_device):
    # variance zero: hat = 0, and the gradient is scaled by 1 / sqrt(eps)
    check_rows = 6
    desc = jfa.make_block_norm(rows=check_rows, dim=48, dtype="f32", post_norm="layer", pre_norm="layer", gate="none")
    x = torch.zeros(check_rows, 48)
    b = torch.full((check_rows, 48), 3.0)
    dy, dn = torch.randn(check_rows, 48), torch.randn(check_rows, 48)
    d = lambda t: t.to(cuda_device)
    y, n = jfa.block_norm_forward(desc, d(x), d(b))
    assert (y == 0).all() and (n == 0).all()
    g = jfa.block_norm_backward(desc, d(x), d(b), dy=d(dy), dn=d(dn))
    ref = mx4.block_norm(x.numpy(), b.numpy(), post="layer", pre="layer", gate_kind="none", eps=np.float32(1e-5),
                         dy=dy.numpy(), dn=dn.numpy())
    for name in ("x", "block"):
        close(g[name], ref[name], 340, name)


def test_no_rows(cuda_device):
    desc = jfa.make_block_norm(rows=0, dim=40)
    x = torch.zeros(0, 40, dtype=torch.bfloat16, device=cuda_device)
    p = torch.ones(40, device=cuda_device)
    y, n = jfa.block_norm_forward(desc, x, x, x, scale=p, post_gamma=p, pre_gamma=p)
    assert y.shape == n.shape == (0, 40)
    g = jfa.block_norm_backward(desc, x, x, x, scale=p, post_gamma=p, pre_gamma=p, dy=x, dn=x)
    for name in ("scale", "post_gamma", "pre_gamma"):
        assert torch.equal(g[name], torch.zeros(40, device=cuda_device))


def test_writes_its_rows_only_and_repeats(cuda_device):
    for rows, dim in ((5, 100), (9, 104)):
        kw, up = make(rows, dim, "bf16", "rms", "rms", "silu")
        kw, up = dev_(kw, cuda_device), dev_(up, cuda_device)
        desc = jfa.make_block_norm(rows=rows, dim=dim)
        y, n = jfa.block_norm_forward(desc, **kw)
        g = jfa.block_norm_backward(desc, **kw, **up)
        g2 = jfa.block_norm_backward(desc, **kw, **up)
        assert all(torch.equal(g[k], g2[k]) for k in g if g[k] is not None)
        big = [torch.full((rows * dim + 64,), 7.0, dtype=torch.bfloat16, device=cuda_device) for _ in range(5)]
        sums = [torch.full((dim + 16,), 7.0, device=cuda_device) for _ in range(3)]
        jfa.jfa_block_norm_forward(desc, *kw.values(), big[0], big[1])
        jfa.jfa_block_norm_backward(desc, *kw.values(), up["dy"], up["dn"], big[2], big[3], big[4], sums[0], sums[1],
                                    None, sums[2], None, jfa.block_norm_workspace(desc, cuda_device))
        for got, ref in zip(big, (y, n, g["x"], g["block"], g["gate"])):
            assert torch.equal(got[:rows * dim].reshape(rows, dim), ref) and (got[rows * dim:] == 7.0).all()
        for got, ref in zip(sums, (g["scale"], g["post_gamma"], g["pre_gamma"])):
            assert torch.equal(got[:dim], ref) and (got[dim:] == 7.0).all()


def test_graph_capture_and_streams(cuda_device):
    desc = jfa.make_block_norm(rows=300, dim=264)
    sets = [tuple(dev_(t, cuda_device) for t in make(300, 264, "bf16", "rms", "rms", "silu", seed=s)) for s in range(3)]
    want = [(jfa.block_norm_forward(desc, **kw), jfa.block_norm_backward(desc, **kw, **up)) for kw, up in sets]
    side = torch.cuda.Stream(cuda_device)
    torch.cuda.synchronize()
    (y, n), g = (jfa.block_norm_forward(desc, **sets[0][0], stream=side),
                 jfa.block_norm_backward(desc, **sets[0][0], **sets[0][1], stream=side))
    torch.cuda.synchronize()
    assert torch.equal(y, want[0][0][0]) and all(torch.equal(g[k], want[0][1][k]) for k in g if g[k] is not None)
    kw, up = ({k: None if t is None else t.clone() for k, t in s.items()} for s in sets[0])
    ws = jfa.block_norm_workspace(desc, cuda_device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, n = jfa.block_norm_forward(desc, **kw)
        g = jfa.block_norm_backward(desc, **kw, **up, ws=ws)
    for (kw_s, up_s), ((y_r, n_r), g_r) in zip(sets, want):
        for dst, src in ((kw, kw_s), (up, up_s)):
            for k in dst:
                if dst[k] is not None:
                    dst[k].copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y_r) and torch.equal(n, n_r)
        assert all(torch.equal(g[k], g_r[k]) for k in g if g[k] is not None)


@pytest.mark.parametrize("dim", [64, 101, 1024, 1027])
def test_bad_values_stay_in_their_row(cuda_device, dim):
    kw, up = make(9, dim, "bf16", "rms", "layer", "silu", seed=1)
    kw, up = dev_(kw, cuda_device), dev_(up, cuda_device)
    desc = jfa.make_block_norm(rows=9, dim=dim, post_norm="rms", pre_norm="layer")
    y, n = jfa.block_norm_forward(desc, **kw)
    g = jfa.block_norm_backward(desc, **kw, **up)
    for where, value in (("block", float("nan")), ("x", float("inf")), ("gate", float("-inf"))):
        bad = {k: None if t is None else t.clone() for k, t in kw.items()}
        bad[where][4, dim - 1] = value
        by, bn = jfa.block_norm_forward(desc, **bad)
        bg = jfa.block_norm_backward(desc, **bad, **up)
        keep = [i for i in range(9) if i != 4]
        assert torch.equal(by[keep], y[keep]) and torch.equal(bn[keep], n[keep])
        assert all(torch.equal(bg[k][keep], g[k][keep]) for k in ("x", "block", "gate"))
        assert torch.isnan(bn[4]).any()


def test_offsets_past_32_bits(cuda_device):
    # 2.3e9 elements: the last rows against the same rows alone
    rows, dim = 2_240_001, 1024
    x, b, u = (torch.empty(rows, dim, dtype=torch.bfloat16, device=cuda_device) for _ in range(3))
    for i, t in enumerate((x, b, u)):
        t[-64:] = torch.randn(64, dim, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).to(cuda_device)
        t[:-64] = 0
    p = torch.ones(dim, device=cuda_device)
    kw = dict(scale=p, post_gamma=p, pre_gamma=p)
    y, n = jfa.block_norm_forward(jfa.make_block_norm(rows=rows, dim=dim), x, b, u, **kw)
    small = jfa.make_block_norm(rows=64, dim=dim)
    cut = [t[-64:].clone() for t in (x, b, u)]
    ys, ns = jfa.block_norm_forward(small, *cut, **kw)
    assert torch.equal(y[-64:], ys) and torch.equal(n[-64:], ns) and (y[:-64] == 0).all()
    del y, n
    g = jfa.block_norm_backward(jfa.make_block_norm(rows=rows, dim=dim), x, b, u, dy=x, dn=b, **kw)
    gs = jfa.block_norm_backward(small, *cut, dy=cut[0], dn=cut[1], **kw)
    for k in ("x", "block", "gate"):
        assert torch.equal(g[k][-64:], gs[k])
