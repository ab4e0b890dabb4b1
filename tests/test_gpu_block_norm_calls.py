"""The block norms on the GPU: host threads side by side, rows of one number."""
import ctypes
import sys
import threading

import numpy as np
import pytest
import torch

from jagged_attention_recommender_jfa_b200 import jfa
from test_gpu_block_norm import TORCH, dev_, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,narrow,wide", [("bf16", 2048, 4096), ("f32", 1544, 4096), ("bf16", 4500, 6144)])
def test_host_threads_with_widths_of_one_kernel(cuda_device, dtype, narrow, wide):
    # widths that share a kernel and ask for different amounts of shared memory,
    # from host threads and streams of their own: every call is accepted and
    # gives the bits of a lone call
    rows, lib = 300, jfa.load()

    def caller(dim):
        kw, up = make(rows, dim, dtype, "layer", "layer", "silu", seed=dim)
        kw, up = dev_(kw, cuda_device), dev_(up, cuda_device)
        desc = jfa.make_block_norm(rows=rows, dim=dim, dtype=dtype, post_norm="layer", pre_norm="layer")
        want = jfa.block_norm_backward(desc, **kw, **up)
        got = {k: torch.zeros_like(t) for k, t in want.items()}
        ws, stream = jfa.block_norm_workspace(desc, cuda_device), torch.cuda.Stream(cuda_device)
        args = [t.data_ptr() for t in (*kw.values(), *up.values(), *got.values(), ws)]

        def run():   # converted once, so that the loop is little more than the library's own time
            for _ in range(1500):
                status.append(lib.jfa_block_norm_backward(ctypes.byref(desc), *args, ws.numel(), stream.cuda_stream))

        status = []
        return run, status, want, got, (kw, up, ws)

    callers = [caller(d) for d in (narrow, wide, narrow, wide)]
    torch.cuda.synchronize()
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=c[0]) for c in callers]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    for _, status, want, got, _ in callers:
        assert len(status) == 1500 and not any(status), (sum(map(bool, status)), max(status))
        assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,value", [(1000, 1000.0), (1003, 24.0), (48, -7.0), (5000, 512.0), (7, 3.0)])
def test_constant_stream_is_centred_to_zero(cuda_device, dtype, dim, value):
    # y is one number throughout a row and its sums are whole numbers below
    # 2^24, so its mean is exact: n is beta and dgamma zero, whatever 1 / D rounds to
    x = torch.full((5, dim), value, dtype=TORCH[dtype], device=cuda_device)
    zero = torch.zeros_like(x)
    up = torch.from_numpy(np.random.default_rng(dim).normal(size=(5, dim))).to(x)
    beta = torch.arange(dim, dtype=torch.float32, device=cuda_device)
    gamma = torch.full_like(beta, 2.0)
    assert abs(value) * dim < 2 ** 24
    for post in ("none", "rms", "layer"):
        desc = jfa.make_block_norm(rows=5, dim=dim, dtype=dtype, post_norm=post, pre_norm="layer", gate="none", eps=1e-6)
        y, n = jfa.block_norm_forward(desc, x, zero, pre_gamma=gamma, pre_beta=beta)
        assert torch.equal(y, x)
        assert torch.equal(n, beta.to(x.dtype).expand(5, dim)), (post, (n - beta).abs().max())
        g = jfa.block_norm_backward(desc, x, zero, pre_gamma=gamma, pre_beta=beta, dy=up, dn=up)
        assert (g["pre_gamma"] == 0).all(), post
