"""Calls of the block norms on the GPU from host threads side by side."""
import ctypes
import sys
import threading

import pytest
import torch

from jagged_attention_recommender_jfa_b200 import jfa
from test_gpu_block_norm import dev_, make

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
