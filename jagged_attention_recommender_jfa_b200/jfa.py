"""Python binding of libjfa (ctypes).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libjfa.so``.  The functions named like the C entry points
(``jfa_forward``, ``jfa_backward``, ...) take torch tensors (device memory)
or raw integer addresses and raise :class:`JfaError` on a non-OK status.
``attention_forward`` / ``attention_backward`` additionally allocate outputs
and the workspace with torch.

If ``libjfa.so`` is missing it is built with nvcc (the same sm_100a build as
``python -m jagged_attention_recommender_jfa_b200.build``); if that is not
possible the import of the library fails loudly -- there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libjfa.so")
_LOCK = threading.Lock()
_LIB = None

JFA_OK, JFA_ERR_INVALID_ARGUMENT, JFA_ERR_UNSUPPORTED, JFA_ERR_WORKSPACE = 0, 1, 2, 3
JFA_ERR_CUDA, JFA_ERR_TIMEOUT, JFA_ERR_BAD_OFFSETS = 4, 5, 6
JFA_F32, JFA_BF16, JFA_MXFP8 = 0, 1, 2
ACT = {"softmax": 0, "silu": 1, "gelu_tanh": 2}
BIAS = {"none": 0, "relpos": 1, "dense": 2}
DTYPE = {"f32": JFA_F32, "bf16": JFA_BF16, "mxfp8": JFA_MXFP8}
STATUS_NAMES = {0: "JFA_OK", 1: "JFA_ERR_INVALID_ARGUMENT", 2: "JFA_ERR_UNSUPPORTED",
                3: "JFA_ERR_WORKSPACE", 4: "JFA_ERR_CUDA", 5: "JFA_ERR_TIMEOUT",
                6: "JFA_ERR_BAD_OFFSETS"}

# Every symbol include/jfa.h declares.
EXPORTS = ("jfa_workspace_bytes", "jfa_forward", "jfa_backward", "jfa_quantize_mxfp8",
           "jfa_quantize_mxfp8_dequant",
           "jfa_schedule", "jfa_check_error", "jfa_last_error", "jfa_path",
           "jfa_profile_enable", "jfa_profile_read", "jfa_kernel_name",
           "jfa_forward_fixed_scratch", "jfa_partition", "jfa_backward_dbias",
           "jfa_block_offsets", "jfa_test_inject", "jfa_forward_mxfp8",
           "jfa_norm_quantize_mxfp8", "jfa_mxfp4_code_bytes", "jfa_mxfp4_scale_bytes",
           "jfa_mxfp4_workspace_bytes", "jfa_quantize_mxfp4", "jfa_quantize_mxfp4_dequant",
           "jfa_quantize_mxfp4_both",
           "jfa_matmul_mxfp4", "jfa_linear_mxfp4_scratch_bytes", "jfa_linear_mxfp4_forward",
           "jfa_linear_mxfp4_backward", "jfa_block_norm_workspace_bytes", "jfa_block_norm_forward",
           "jfa_block_norm_backward")
NORM = {"none": 0, "rms": 1, "layer": 2}
GATE = {"none": 0, "identity": 1, "silu": 2, "sigmoid": 3}
JFA_TEST_FWD_SKIP_LOAD, JFA_TEST_MATMUL_SKIP_LOAD = 1, 2
PARTITION = {"lpt": 0, "bbs": 1}


class JfaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class jfa_problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("max_q_len", ctypes.c_int32),
                ("max_kv_len", ctypes.c_int32), ("total_q", ctypes.c_int64),
                ("total_kv", ctypes.c_int64), ("dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("bias_kind", ctypes.c_int), ("relpos_len", ctypes.c_int32),
                ("window", ctypes.c_int32)]


class jfa_block_norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("post_norm", ctypes.c_int), ("pre_norm", ctypes.c_int), ("gate", ctypes.c_int),
                ("eps", ctypes.c_float)]


class MxOperand(NamedTuple):
    """An MXFP4 operand of ``rows`` x ``cols`` (layouts in jfa.h)."""
    codes: torch.Tensor    # uint8 [rows][ceil(cols / 32) * 16]
    scales: torch.Tensor   # uint8, 128 x 4 tiles
    rows: int
    cols: int


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Loads libjfa.so (building it if absent) and declares the signatures."""
    global _LIB
    if _LIB is not None:
        return _LIB
    with _LOCK:
        if _LIB is not None:
            return _LIB
        if not os.path.exists(_LIB_PATH):
            from . import build as _build
            _build.build()
        lib = ctypes.CDLL(_LIB_PATH)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        PP = ctypes.POINTER(jfa_problem)
        lib.jfa_workspace_bytes.argtypes = [PP, i32]
        lib.jfa_workspace_bytes.restype = sz
        lib.jfa_forward.argtypes = [PP, P, P, P, P, P, P, i32, i32, P, P, P, sz, P]
        lib.jfa_forward.restype = i32
        lib.jfa_backward.argtypes = [PP, P, P, P, P, P, P, P, P, P, i32, i32, P, P, P, P, sz, P]
        lib.jfa_backward.restype = i32
        lib.jfa_quantize_mxfp8.argtypes = [P, i64, i32, i32, P, i32, i32, i32, P, P, P]
        lib.jfa_quantize_mxfp8.restype = i32
        lib.jfa_quantize_mxfp8_dequant.argtypes = [P, i64, i32, i32, P, i32, i32, i32, P, P, P, P]
        lib.jfa_quantize_mxfp8_dequant.restype = i32
        lib.jfa_schedule.argtypes = [PP, P, P, i32, i32, i32, P, i64, P, P, sz, P]
        lib.jfa_schedule.restype = i32
        lib.jfa_check_error.argtypes = [P, P]
        lib.jfa_check_error.restype = i32
        lib.jfa_last_error.restype = ctypes.c_char_p
        lib.jfa_path.argtypes = [PP, i32, i32]
        lib.jfa_path.restype = i32
        lib.jfa_profile_enable.argtypes = [i32]
        lib.jfa_profile_enable.restype = i32
        lib.jfa_profile_read.argtypes = [P, P, i32]
        lib.jfa_profile_read.restype = i32
        lib.jfa_kernel_name.argtypes = [i32]
        lib.jfa_kernel_name.restype = ctypes.c_char_p
        lib.jfa_forward_fixed_scratch.argtypes = [PP, P, P, P, P, P, P, i32, i32, P, P, P]
        lib.jfa_forward_fixed_scratch.restype = i32
        lib.jfa_backward_dbias.argtypes = [PP, P, P, P, P, P, P, P, P, P, i32, i32, P, P, P, P, P,
                                           sz, P]
        lib.jfa_backward_dbias.restype = i32
        lib.jfa_forward_mxfp8.argtypes = [PP, P, P, P, P, P, P, P, P, P, i32, P, P, P, sz, P]
        lib.jfa_forward_mxfp8.restype = i32
        lib.jfa_norm_quantize_mxfp8.argtypes = [P, i64, i32, P, P, ctypes.c_float, i32, P, P, P]
        lib.jfa_norm_quantize_mxfp8.restype = i32
        for name in ("jfa_mxfp4_code_bytes", "jfa_mxfp4_scale_bytes"):
            getattr(lib, name).argtypes = [i64, i64]
            getattr(lib, name).restype = sz
        lib.jfa_mxfp4_workspace_bytes.argtypes = []
        lib.jfa_mxfp4_workspace_bytes.restype = sz
        lib.jfa_quantize_mxfp4.argtypes = [P, i32, i64, i64, i32, P, P, P]
        lib.jfa_quantize_mxfp4.restype = i32
        lib.jfa_quantize_mxfp4_dequant.argtypes = [P, i32, i64, i64, i32, P, P, P, P]
        lib.jfa_quantize_mxfp4_dequant.restype = i32
        lib.jfa_quantize_mxfp4_both.argtypes = [P, i32, i64, i64, P, P, P, P, P]
        lib.jfa_quantize_mxfp4_both.restype = i32
        lib.jfa_matmul_mxfp4.argtypes = [i64, i64, i64, P, P, P, P, P, P, i32, i32, P, sz, P]
        lib.jfa_matmul_mxfp4.restype = i32
        lib.jfa_linear_mxfp4_scratch_bytes.argtypes = [i64, i64, i64, i32]
        lib.jfa_linear_mxfp4_scratch_bytes.restype = sz
        lib.jfa_linear_mxfp4_forward.argtypes = [P, i32, i64, i64, i64, P, P, P, P, P, sz, P, sz, P]
        lib.jfa_linear_mxfp4_forward.restype = i32
        lib.jfa_linear_mxfp4_backward.argtypes = [P, i32, P, i32, i64, i64, i64, P, P, P, P, i32, P, sz,
                                                  P, sz, P]
        lib.jfa_linear_mxfp4_backward.restype = i32
        PN = ctypes.POINTER(jfa_block_norm)
        lib.jfa_block_norm_workspace_bytes.argtypes = [PN]
        lib.jfa_block_norm_workspace_bytes.restype = sz
        lib.jfa_block_norm_forward.argtypes = [PN] + [P] * 11
        lib.jfa_block_norm_forward.restype = i32
        lib.jfa_block_norm_backward.argtypes = [PN] + [P] * 19 + [sz, P]
        lib.jfa_block_norm_backward.restype = i32
        lib.jfa_test_inject.argtypes = [i32]
        lib.jfa_test_inject.restype = i32
        lib.jfa_block_offsets.argtypes = [P, i32, i64, i32, P, P]
        lib.jfa_block_offsets.restype = i32
        lib.jfa_partition.argtypes = [i32, P, P, i32, i32, i32, i32, i32, P, P]
        lib.jfa_partition.restype = i32
        _LIB = lib
        return lib


def _addr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        return x.data_ptr() if x.numel() > 0 else None
    return int(x)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int):
    if status != JFA_OK:
        raise JfaError(status, load().jfa_last_error().decode())


def make_problem(*, batch, heads, head_dim, max_q_len, max_kv_len, total_q, total_kv,
                 dtype="bf16", scale=0.0, bias_kind="none", relpos_len=0, window=0) -> jfa_problem:
    """``window`` > 0: sliding window of that width (0: none)."""
    return jfa_problem(int(batch), int(heads), int(head_dim), int(max_q_len), int(max_kv_len),
                       int(total_q), int(total_kv), DTYPE[dtype] if isinstance(dtype, str) else int(dtype),
                       float(scale), BIAS[bias_kind] if isinstance(bias_kind, str) else int(bias_kind),
                       int(relpos_len), int(window))


def problem_of(p, dtype: Optional[str] = None, window: int = 0) -> jfa_problem:
    """Descriptor of an ``inputs.Problem`` batch."""
    return make_problem(batch=p.B, heads=p.H, head_dim=p.d, max_q_len=p.max_q_len,
                        max_kv_len=p.max_kv_len, total_q=p.total_q, total_kv=p.total_kv,
                        dtype=dtype or p.dtype, bias_kind=p.bias_kind, relpos_len=p.relpos_len,
                        window=window)


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def jfa_workspace_bytes(problem: jfa_problem, backward: int) -> int:
    return int(load().jfa_workspace_bytes(ctypes.byref(problem), int(backward)))


def jfa_path(problem: jfa_problem, act, backward: int) -> int:
    return int(load().jfa_path(ctypes.byref(problem), ACT.get(act, act), int(backward)))


def jfa_forward(problem, q, k, v, q_offsets, kv_offsets, bias, act, causal, out, lse, workspace,
                ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().jfa_forward(ctypes.byref(problem), _addr(q), _addr(k), _addr(v),
                              _addr(q_offsets), _addr(kv_offsets), _addr(bias),
                              ACT.get(act, act), int(bool(causal)), _addr(out), _addr(lse),
                              _addr(workspace), int(ws_bytes), _stream(stream)))


def jfa_forward_mxfp8(problem, q8, q_scales, k8, k_scales, v8, v_scales, q_offsets, kv_offsets,
                      bias, causal, out, lse, workspace, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().jfa_forward_mxfp8(ctypes.byref(problem), _addr(q8), _addr(q_scales), _addr(k8),
                                    _addr(k_scales), _addr(v8), _addr(v_scales), _addr(q_offsets),
                                    _addr(kv_offsets), _addr(bias), int(bool(causal)), _addr(out),
                                    _addr(lse), _addr(workspace), int(ws_bytes), _stream(stream)))


def jfa_forward_fixed_scratch(problem, q, k, v, q_offsets, kv_offsets, bias, act, causal, out,
                              lse, stream=None):
    """Forward without a workspace: for callers that cannot allocate device
    memory (scratch is a fixed 8 MiB array inside the library; see jfa.h)."""
    _check(load().jfa_forward_fixed_scratch(ctypes.byref(problem), _addr(q), _addr(k), _addr(v),
                                            _addr(q_offsets), _addr(kv_offsets), _addr(bias),
                                            ACT.get(act, act), int(bool(causal)), _addr(out),
                                            _addr(lse), _stream(stream)))


def jfa_backward(problem, q, k, v, out, lse, dout, q_offsets, kv_offsets, bias, act, causal,
                 dq, dk, dv, workspace, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().jfa_backward(ctypes.byref(problem), _addr(q), _addr(k), _addr(v), _addr(out),
                               _addr(lse), _addr(dout), _addr(q_offsets), _addr(kv_offsets),
                               _addr(bias), ACT.get(act, act), int(bool(causal)), _addr(dq),
                               _addr(dk), _addr(dv), _addr(workspace), int(ws_bytes),
                               _stream(stream)))


def jfa_backward_dbias(problem, q, k, v, out, lse, dout, q_offsets, kv_offsets, bias, act,
                       causal, dq, dk, dv, dbias, workspace, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().jfa_backward_dbias(ctypes.byref(problem), _addr(q), _addr(k), _addr(v),
                                     _addr(out), _addr(lse), _addr(dout), _addr(q_offsets),
                                     _addr(kv_offsets), _addr(bias), ACT.get(act, act),
                                     int(bool(causal)), _addr(dq), _addr(dk), _addr(dv),
                                     _addr(dbias), _addr(workspace), int(ws_bytes),
                                     _stream(stream)))


def jfa_quantize_mxfp8(x, rows, heads, d, offsets, batch, max_len, along_rows, codes, scales,
                       stream=None):
    _check(load().jfa_quantize_mxfp8(_addr(x), int(rows), int(heads), int(d), _addr(offsets),
                                     int(batch), int(max_len), int(bool(along_rows)),
                                     _addr(codes), _addr(scales), _stream(stream)))


def jfa_quantize_mxfp8_dequant(x, rows, heads, d, offsets, batch, max_len, along_rows, codes,
                               scales, dequant, stream=None):
    _check(load().jfa_quantize_mxfp8_dequant(_addr(x), int(rows), int(heads), int(d), _addr(offsets),
                                             int(batch), int(max_len), int(bool(along_rows)),
                                             _addr(codes), _addr(scales), _addr(dequant),
                                             _stream(stream)))


def jfa_schedule(problem, q_offsets, kv_offsets, causal, backward, tile, items, capacity, count,
                 workspace, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().jfa_schedule(ctypes.byref(problem), _addr(q_offsets), _addr(kv_offsets),
                               int(bool(causal)), int(bool(backward)), int(tile), _addr(items),
                               int(capacity), _addr(count), _addr(workspace), int(ws_bytes),
                               _stream(stream)))


def jfa_block_offsets(offsets, batch, total, block, block_offsets, stream=None):
    _check(load().jfa_block_offsets(_addr(offsets), int(batch), int(total), int(block),
                                    _addr(block_offsets), _stream(stream)))


def block_attention(problem: jfa_problem, offsets, block: int, stream=None):
    """BlockAttention with block length ``block`` as a jagged problem over the
    blocks: returns (descriptor, block offsets) to pass to jfa_forward /
    jfa_backward as both q and kv offsets (self-attention)."""
    n_out = problem.batch + problem.total_q // block
    boff = torch.empty(n_out + 1, dtype=torch.int32, device=offsets.device)
    jfa_block_offsets(offsets, problem.batch, problem.total_q, block, boff, stream)
    p2 = jfa_problem.from_buffer_copy(problem)
    p2.batch = n_out
    p2.max_q_len = min(block, problem.max_q_len)
    p2.max_kv_len = min(block, problem.max_kv_len)
    return p2, boff


def jfa_partition(q_lens, kv_lens, causal, ranks, method="lpt", sub_batch=1, window=0):
    """Host-side split of a global batch across ``ranks``: returns (rank_of
    int32 [batch], rank_cost int64 [ranks]) as numpy arrays.  ``window`` > 0
    counts a sliding window's pairs."""
    import numpy as np
    ql = np.ascontiguousarray(np.asarray(q_lens, np.int32))
    kl = np.ascontiguousarray(np.asarray(kv_lens, np.int32))
    assert ql.shape == kl.shape and ql.ndim == 1
    rank_of = np.zeros(len(ql), np.int32)
    rank_cost = np.zeros(int(ranks), np.int64)
    c = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(load().jfa_partition(len(ql), c(ql), c(kl), int(bool(causal)), int(window), int(ranks),
                                PARTITION.get(method, method), int(sub_batch), c(rank_of),
                                c(rank_cost)))
    return rank_of, rank_cost


def jfa_norm_quantize_mxfp8(x, rows, D, gamma, beta, eps, layernorm, codes, scales, stream=None):
    _check(load().jfa_norm_quantize_mxfp8(_addr(x), int(rows), int(D), _addr(gamma), _addr(beta),
                                          float(eps), int(bool(layernorm)), _addr(codes),
                                          _addr(scales), _stream(stream)))


def jfa_mxfp4_code_bytes(rows, cols) -> int:
    return int(load().jfa_mxfp4_code_bytes(int(rows), int(cols)))


def jfa_mxfp4_scale_bytes(rows, cols) -> int:
    return int(load().jfa_mxfp4_scale_bytes(int(rows), int(cols)))


def jfa_mxfp4_workspace_bytes() -> int:
    return int(load().jfa_mxfp4_workspace_bytes())


def jfa_quantize_mxfp4(x, dtype, rows, cols, along_rows, codes, scales, stream=None):
    _check(load().jfa_quantize_mxfp4(_addr(x), DTYPE.get(dtype, dtype), int(rows), int(cols),
                                     int(bool(along_rows)), _addr(codes), _addr(scales),
                                     _stream(stream)))


def jfa_quantize_mxfp4_dequant(x, dtype, rows, cols, along_rows, codes, scales, dequant,
                               stream=None):
    _check(load().jfa_quantize_mxfp4_dequant(_addr(x), DTYPE.get(dtype, dtype), int(rows),
                                             int(cols), int(bool(along_rows)), _addr(codes),
                                             _addr(scales), _addr(dequant), _stream(stream)))


def jfa_quantize_mxfp4_both(x, dtype, rows, cols, codes, scales, codes_t, scales_t, stream=None):
    _check(load().jfa_quantize_mxfp4_both(_addr(x), DTYPE.get(dtype, dtype), int(rows), int(cols),
                                          _addr(codes), _addr(scales), _addr(codes_t),
                                          _addr(scales_t), _stream(stream)))


def _nbytes(t, given=None) -> int:
    """The bytes behind a buffer's address.  A strided or expanded tensor does
    not have the memory that its element count says."""
    if given is not None:
        return int(given)
    if not isinstance(t, torch.Tensor) or not t.is_contiguous():
        _invalid("a workspace or scratch buffer must be a contiguous tensor, or its size be given")
    return t.numel() * t.element_size()


def jfa_matmul_mxfp4(m, n, k, a_codes, a_scales, b_codes, b_scales, bias, out, out_dtype,
                     accumulate, workspace, ws_bytes=None, stream=None):
    _check(load().jfa_matmul_mxfp4(int(m), int(n), int(k), _addr(a_codes), _addr(a_scales),
                                   _addr(b_codes), _addr(b_scales), _addr(bias), _addr(out),
                                   DTYPE.get(out_dtype, out_dtype), int(bool(accumulate)),
                                   _addr(workspace), _nbytes(workspace, ws_bytes), _stream(stream)))


def jfa_linear_mxfp4_scratch_bytes(m, n, k, backward) -> int:
    return int(load().jfa_linear_mxfp4_scratch_bytes(int(m), int(n), int(k), int(bool(backward))))


def jfa_linear_mxfp4_forward(x, dtype, m, n, k, w_codes, w_scales, bias, y, scratch, workspace,
                             scratch_bytes=None, ws_bytes=None, stream=None):
    _check(load().jfa_linear_mxfp4_forward(_addr(x), DTYPE.get(dtype, dtype), int(m), int(n), int(k),
                                           _addr(w_codes), _addr(w_scales), _addr(bias), _addr(y),
                                           _addr(scratch), _nbytes(scratch, scratch_bytes),
                                           _addr(workspace), _nbytes(workspace, ws_bytes),
                                           _stream(stream)))


def jfa_linear_mxfp4_backward(dy, dtype, x, x_dtype, m, n, k, wt_codes, wt_scales, dx, dw, accumulate,
                              scratch, workspace, scratch_bytes=None, ws_bytes=None, stream=None):
    _check(load().jfa_linear_mxfp4_backward(_addr(dy), DTYPE.get(dtype, dtype), _addr(x),
                                            DTYPE.get(x_dtype, x_dtype), int(m), int(n), int(k),
                                            _addr(wt_codes), _addr(wt_scales), _addr(dx), _addr(dw),
                                            int(bool(accumulate)), _addr(scratch),
                                            _nbytes(scratch, scratch_bytes), _addr(workspace),
                                            _nbytes(workspace, ws_bytes), _stream(stream)))


def make_block_norm(*, rows, dim, dtype="bf16", post_norm="rms", pre_norm="rms", gate="silu",
                    eps=1e-5) -> jfa_block_norm:
    return jfa_block_norm(int(rows), int(dim), DTYPE.get(dtype, dtype),
                          NORM.get(post_norm, post_norm), NORM.get(pre_norm, pre_norm),
                          GATE.get(gate, gate), float(eps))


def jfa_block_norm_workspace_bytes(desc: jfa_block_norm) -> int:
    return int(load().jfa_block_norm_workspace_bytes(ctypes.byref(desc)))


def jfa_block_norm_forward(desc, x, block, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta,
                           y, n, stream=None):
    _check(load().jfa_block_norm_forward(ctypes.byref(desc), _addr(x), _addr(block), _addr(gate),
                                         _addr(scale), _addr(post_gamma), _addr(post_beta),
                                         _addr(pre_gamma), _addr(pre_beta), _addr(y), _addr(n),
                                         _stream(stream)))


def jfa_block_norm_backward(desc, x, block, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta,
                            dy, dn, dx, dblock, dgate, dscale, dpost_gamma, dpost_beta, dpre_gamma,
                            dpre_beta, workspace, ws_bytes=None, stream=None):
    _check(load().jfa_block_norm_backward(ctypes.byref(desc), _addr(x), _addr(block), _addr(gate),
                                          _addr(scale), _addr(post_gamma), _addr(post_beta),
                                          _addr(pre_gamma), _addr(pre_beta), _addr(dy), _addr(dn),
                                          _addr(dx), _addr(dblock), _addr(dgate), _addr(dscale),
                                          _addr(dpost_gamma), _addr(dpost_beta), _addr(dpre_gamma),
                                          _addr(dpre_beta), _addr(workspace),
                                          _nbytes(workspace, ws_bytes), _stream(stream)))


def jfa_test_inject(what: int):
    _check(load().jfa_test_inject(int(what)))


def jfa_profile_enable(enable: bool):
    _check(load().jfa_profile_enable(int(bool(enable))))


def jfa_profile_read():
    """[(kernel name, ms), ...] of the launches recorded since profiling was enabled."""
    lib = load()
    n = lib.jfa_profile_read(None, None, 0)
    if n < 0:
        raise JfaError(JFA_ERR_CUDA, "profile read failed")
    ms = (ctypes.c_float * max(n, 1))()
    ids = (ctypes.c_int32 * max(n, 1))()
    n2 = lib.jfa_profile_read(ms, ids, n)
    if n2 < 0:
        raise JfaError(JFA_ERR_CUDA, "profile read failed")
    return [(lib.jfa_kernel_name(ids[i]).decode(), float(ms[i])) for i in range(n)]


def jfa_kernel_name(kernel_id: int) -> str:
    return load().jfa_kernel_name(int(kernel_id)).decode()


def jfa_check_error(workspace, stream=None):
    _check(load().jfa_check_error(_addr(workspace), _stream(stream)))


# ---------------------------------------------------------------------------
# Allocating conveniences (torch owns the memory)
# ---------------------------------------------------------------------------

def workspace(problem: jfa_problem, backward: bool, device) -> torch.Tensor:
    n = jfa_workspace_bytes(problem, int(backward))
    if n == 0:
        raise JfaError(JFA_ERR_INVALID_ARGUMENT, load().jfa_last_error().decode())
    return torch.empty(n, dtype=torch.uint8, device=device)


def attention_forward(problem, q, k, v, q_offsets, kv_offsets, bias=None, act="softmax",
                      causal=False, ws=None, stream=None, check=True):
    """Allocates out / lse (and the workspace unless ``ws`` is given) and runs
    jfa_forward.  With ``check`` (the default) the stream is synchronised and
    the workspace's device error word is read, so that bad offsets or a timed
    out device wait raise :class:`JfaError` here; ``check=False`` leaves that
    to the caller (``jfa_check_error(ws)``) and keeps the call asynchronous."""
    out = torch.empty_like(q)
    lse = None
    if act == "softmax":
        lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(problem, False, q.device)
    jfa_forward(problem, q, k, v, q_offsets, kv_offsets, bias, act, causal, out, lse, ws,
                stream=stream)
    if check:
        jfa_check_error(ws, stream)
    return out, lse


def attention_backward(problem, q, k, v, out, lse, dout, q_offsets, kv_offsets, bias=None,
                       act="softmax", causal=False, ws=None, stream=None, check=True,
                       want_dbias=False):
    """Allocates dq / dk / dv (and the workspace unless ``ws`` is given) and
    runs jfa_backward; ``check`` as in :func:`attention_forward`.  With
    ``want_dbias`` it runs jfa_backward_dbias and also returns the bias
    gradient (shaped like ``bias``)."""
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if ws is None:
        ws = workspace(problem, True, q.device)
    if want_dbias:
        dbias = torch.empty_like(bias)
        jfa_backward_dbias(problem, q, k, v, out, lse, dout, q_offsets, kv_offsets, bias, act,
                           causal, dq, dk, dv, dbias, ws, stream=stream)
    else:
        jfa_backward(problem, q, k, v, out, lse, dout, q_offsets, kv_offsets, bias, act, causal,
                     dq, dk, dv, ws, stream=stream)
    if check:
        jfa_check_error(ws, stream)
    return (dq, dk, dv, dbias) if want_dbias else (dq, dk, dv)


# ---------------------------------------------------------------------------
# Around the attention: MXFP4 operands and products, block norms.  These take
# contiguous tensors, run on the tensors' own device and, unless ``stream``
# says otherwise, on that device's current stream; with ``stream`` the results
# are allocated on it too.  Their small calls are launches of a few
# microseconds, so the way to them is kept short: arguments are looked over by
# one expression each, and only a call that fails it is taken apart for its
# message.
# ---------------------------------------------------------------------------

_TORCH_DTYPE = {torch.float32: JFA_F32, torch.bfloat16: JFA_BF16}
_JFA_DTYPE = {v: k for k, v in _TORCH_DTYPE.items()}
_U8 = torch.uint8
# the current device, and its current stream's handle without a Stream object
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _invalid(msg: str):
    raise JfaError(JFA_ERR_INVALID_ARGUMENT, msg)


def _is(t, shape, dtype, index):
    """Whether t is a contiguous tensor of the shape and dtype on that GPU."""
    return (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
            and t.get_device() == index and t.is_contiguous())


def _refuse(t, name, shape, dtypes, index=None):
    """Says what is wrong with an argument (nothing happens if it is right)."""
    if not isinstance(t, torch.Tensor):
        _invalid(f"{name}: a torch tensor is needed")
    if t.shape != tuple(shape):
        _invalid(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        _invalid(f"{name}: dtype {t.dtype} is not one of {tuple(dtypes)}")
    if not t.is_cuda or (index is not None and t.get_device() != index):
        _invalid(f"{name}: device {t.device}, expected {'cuda' if index is None else f'cuda:{index}'}")
    if not t.is_contiguous():
        _invalid(f"{name}: must be contiguous")


def _matrix(x, name="x"):
    """Rows and columns of a contiguous bf16 or fp32 matrix on a GPU."""
    if not (isinstance(x, torch.Tensor) and x.dim() == 2 and x.is_cuda and x.dtype in _TORCH_DTYPE
            and x.is_contiguous()):
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            _invalid(f"{name}: a 2-D torch tensor is needed")
        _refuse(x, name, x.shape, _TORCH_DTYPE)
    return x.shape


def _stream_here(index, stream):
    """The handle of the stream to use as things stand, or None where the
    device or the current stream has to be switched first (:func:`_switch`)."""
    return _raw_stream(index) if stream is None and _device() == index else None


@contextlib.contextmanager
def _switch(device, stream):
    """Makes ``device`` and, where given, ``stream`` (a Stream or a handle) the
    current ones."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream is not None and stream.device != device:
        _invalid(f"stream of {stream.device} for tensors of {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def mxfp4_workspace(device) -> torch.Tensor:
    """The zeroed workspace of :func:`matmul_mxfp4` and the linear layer: an
    error word, for one stream's calls.  Calls of several streams may share one
    only with ``check=False`` and one ``jfa_check_error(ws)`` after all of them
    have completed; what that raises concerns them all."""
    return torch.zeros(jfa_mxfp4_workspace_bytes(), dtype=_U8, device=device)


def _code_pitch(cols):
    return (cols + 31) // 32 * 16


def _scale_bytes(rows, cols):
    return (rows + 127) // 128 * ((cols + 127) // 128) * 512


def quantize_mxfp4(x, along_rows=False, want_dequant=False, stream=None):
    """MXFP4 operand of ``x`` [rows, cols] (bf16 or fp32), or of its transpose
    with ``along_rows`` (blocks of 32 rows).  With ``want_dequant`` also
    returns the values it stands for, laid out like ``x``."""
    rows, cols = _matrix(x)
    s = _stream_here(x.get_device(), stream)
    if s is None:
        with _switch(x.device, stream):
            return quantize_mxfp4(x, along_rows, want_dequant)
    r, c = (cols, rows) if along_rows else (rows, cols)
    dev = x.device
    codes = torch.empty(r, _code_pitch(c), dtype=_U8, device=dev)
    scales = torch.empty(_scale_bytes(r, c), dtype=_U8, device=dev)
    lib = _LIB or load()
    if want_dequant:
        dequant = torch.empty_like(x)
        st = lib.jfa_quantize_mxfp4_dequant(
            x.data_ptr(), _TORCH_DTYPE[x.dtype], rows, cols, 1 if along_rows else 0,
            codes.data_ptr(), scales.data_ptr(), dequant.data_ptr(), s)
        if st:
            _check(st)
        return MxOperand(codes, scales, r, c), dequant
    st = lib.jfa_quantize_mxfp4(x.data_ptr(), _TORCH_DTYPE[x.dtype], rows, cols,
                                1 if along_rows else 0, codes.data_ptr(), scales.data_ptr(), s)
    if st:
        _check(st)
    return MxOperand(codes, scales, r, c)


def quantize_mxfp4_both(x, stream=None):
    """The MXFP4 operands of ``x`` and of its transpose, in one pass."""
    rows, cols = _matrix(x)
    s = _stream_here(x.get_device(), stream)
    if s is None:
        with _switch(x.device, stream):
            return quantize_mxfp4_both(x)
    ops = tuple(MxOperand(torch.empty(r, _code_pitch(c), dtype=_U8, device=x.device),
                          torch.empty(_scale_bytes(r, c), dtype=_U8, device=x.device), r, c)
                for r, c in ((rows, cols), (cols, rows)))
    _check(load().jfa_quantize_mxfp4_both(x.data_ptr(), _TORCH_DTYPE[x.dtype], rows, cols,
                                          *[t.data_ptr() for o in ops for t in o[:2]], s))
    return ops


def _operand(o, name, index=None):
    """The operand's parts; on that GPU, or (index None) on any."""
    if not isinstance(o, MxOperand):
        _invalid(f"{name}: an MxOperand is needed")
    codes, scales, rows, cols = o
    if index is None and isinstance(codes, torch.Tensor):
        index = codes.get_device()
    if not (rows >= 0 and cols >= 0 and _is(codes, (rows, _code_pitch(cols)), _U8, index)
            and _is(scales, (_scale_bytes(rows, cols),), _U8, index) and index >= 0):
        if rows < 0 or cols < 0:
            _invalid(f"{name}: negative size")
        _refuse(codes, name + ".codes", (rows, _code_pitch(cols)), (_U8,), index)
        _refuse(scales, name + ".scales", (_scale_bytes(rows, cols),), (_U8,), index)
    return o


def _vector(t, name, n, index):
    if t is not None and not _is(t, (n,), torch.float32, index):
        _refuse(t, name, (n,), (torch.float32,), index)


def _readable(ws, check):
    """Refuses a call whose error word nobody could read: not read here, and in
    a workspace that is gone when the call returns."""
    if ws is None and not check:
        _invalid("check=False needs ws, whose error word jfa_check_error(ws) reads later")


def _ws_on(ws, index):
    """The caller's workspace, on the GPU, or a fresh one."""
    if ws is None:
        return mxfp4_workspace(torch.device("cuda", index))
    return _buffer(ws, index)


def _buffer(ws, index):
    """A workspace of the caller's: memory of that GPU, all of it behind its address."""
    if not isinstance(ws, torch.Tensor) or not ws.is_contiguous():
        _invalid("ws: a contiguous torch tensor is needed")
    if ws.get_device() != index:
        _invalid(f"ws: device {ws.device}, expected cuda:{index}")
    return ws


def matmul_mxfp4(a: MxOperand, b: MxOperand, bias=None, out=None, out_dtype=torch.bfloat16,
                 accumulate=False, ws=None, stream=None, check=True):
    """``a`` [m, k] times the transpose of ``b`` [n, k] (+ ``bias`` [n] fp32),
    allocated in ``out_dtype`` unless ``out`` is given; ``accumulate`` adds to
    ``out``.  ``ws``: :func:`mxfp4_workspace`; ``check`` as in
    :func:`attention_forward`, and ``check=False`` (what a captured call needs)
    only with ``ws``."""
    _readable(ws, check)
    a_codes, a_scales, m, k = _operand(a, "a")
    index = a_codes.get_device()
    b_codes, b_scales, n, kb = _operand(b, "b", index)
    if k != kb:
        _invalid(f"a has {k} columns, b {kb}")
    _vector(bias, "bias", n, index)
    if out is not None:
        if not (_is(out, (m, n), torch.bfloat16, index) or _is(out, (m, n), torch.float32, index)):
            _refuse(out, "out", (m, n), _TORCH_DTYPE, index)
    elif accumulate:
        _invalid("accumulate needs out")
    elif out_dtype not in _TORCH_DTYPE:
        _invalid(f"out_dtype {out_dtype} is not one of {tuple(_TORCH_DTYPE)}")
    s = _stream_here(index, stream)
    if s is None:
        with _switch(a_codes.device, stream):
            return matmul_mxfp4(a, b, bias, out, out_dtype, accumulate, ws, None, check)
    ws = _ws_on(ws, index)
    if out is None:
        out = torch.empty(m, n, dtype=out_dtype, device=a_codes.device)
    st = (_LIB or load()).jfa_matmul_mxfp4(
        m, n, k, a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(),
        _ptr(bias), out.data_ptr(), _TORCH_DTYPE[out.dtype], 1 if accumulate else 0, ws.data_ptr(),
        ws.numel() * ws.element_size(), s)
    if st:
        _check(st)
    if check:
        jfa_check_error(ws, s)
    return out


def linear_mxfp4_forward(x, w: MxOperand, bias=None, ws=None, stream=None, check=True):
    """``x`` [m, k] (quantised here) times the transpose of the weight operand
    ``w`` [n, k] (``quantize_mxfp4`` of the weight), in the dtype of ``x``;
    ``ws`` and ``check`` as in :func:`matmul_mxfp4`."""
    _readable(ws, check)
    m, k = _matrix(x)
    index = x.get_device()
    w_codes, w_scales, n, kw = _operand(w, "w", index)
    if k != kw:
        _invalid(f"x has {k} columns, w {kw}")
    _vector(bias, "bias", n, index)
    s = _stream_here(index, stream)
    if s is None:
        with _switch(x.device, stream):
            return linear_mxfp4_forward(x, w, bias, ws, None, check)
    ws = _ws_on(ws, index)
    # room for x's codes, then its scales
    buf = torch.empty(m * _code_pitch(k) + _scale_bytes(m, k), dtype=_U8, device=x.device)
    y = torch.empty(m, n, dtype=x.dtype, device=x.device)
    st = (_LIB or load()).jfa_linear_mxfp4_forward(
        x.data_ptr(), _TORCH_DTYPE[x.dtype], m, n, k, w_codes.data_ptr(), w_scales.data_ptr(), _ptr(bias),
        y.data_ptr(), buf.data_ptr(), buf.numel(), ws.data_ptr(), ws.numel() * ws.element_size(), s)
    if st:
        _check(st)
    if check:
        jfa_check_error(ws, s)
    return y


def linear_mxfp4_backward(dy, x, w_t: MxOperand, dw=None, ws=None, stream=None, check=True):
    """Gradients of :func:`linear_mxfp4_forward`: ``dx`` [m, k] in the dtype of
    ``dy`` and ``dw`` [n, k] fp32 (added to ``dw`` where it is given), each a
    product of operands quantised along its own contraction (the quantiser is
    passed straight through).  ``w_t``: ``quantize_mxfp4(weight,
    along_rows=True)``.  The bias's gradient is ``dy.sum(0)``.  ``ws`` and
    ``check`` as in :func:`matmul_mxfp4`."""
    _readable(ws, check)
    m, n = _matrix(dy, "dy")
    mx, k = _matrix(x)
    index = dy.get_device()
    if mx != m or x.get_device() != index:
        _invalid(f"x: {tuple(x.shape)} on {x.device} does not go with dy: {tuple(dy.shape)} on {dy.device}")
    w_codes, w_scales, kw, nw = _operand(w_t, "w_t", index)
    if kw != k or nw != n:
        _invalid(f"w_t is {kw} x {nw}, expected {k} x {n}")
    accumulate = dw is not None
    if accumulate and not _is(dw, (n, k), torch.float32, index):
        _refuse(dw, "dw", (n, k), (torch.float32,), index)
    s = _stream_here(index, stream)
    if s is None:
        with _switch(dy.device, stream):
            return linear_mxfp4_backward(dy, x, w_t, dw, ws, None, check)
    ws = _ws_on(ws, index)
    dev = dy.device
    # room for the operands of dy, of its transpose and of x's
    buf = torch.empty(m * _code_pitch(n) + _scale_bytes(m, n) + (n + k) * _code_pitch(m) + _scale_bytes(n, m)
                      + _scale_bytes(k, m), dtype=_U8, device=dev)
    dx = torch.empty(m, k, dtype=dy.dtype, device=dev)
    if not accumulate:
        dw = torch.empty(n, k, dtype=torch.float32, device=dev)
    st = (_LIB or load()).jfa_linear_mxfp4_backward(
        dy.data_ptr(), _TORCH_DTYPE[dy.dtype], x.data_ptr(), _TORCH_DTYPE[x.dtype], m, n, k,
        w_codes.data_ptr(), w_scales.data_ptr(), dx.data_ptr(), dw.data_ptr(), 1 if accumulate else 0,
        buf.data_ptr(), buf.numel(), ws.data_ptr(), ws.numel() * ws.element_size(), s)
    if st:
        _check(st)
    if check:
        jfa_check_error(ws, s)
    return dx, dw


def block_norm_workspace(desc: jfa_block_norm, device) -> torch.Tensor:
    n = jfa_block_norm_workspace_bytes(desc)
    if n == 0:
        raise JfaError(JFA_ERR_INVALID_ARGUMENT, load().jfa_last_error().decode())
    return torch.empty(n, dtype=_U8, device=device)


_BLOCK_NORM_PARAMS = ("scale", "post_gamma", "post_beta", "pre_gamma", "pre_beta")


def _block_norm_args(desc, tensors, params):
    """Looks the tensors ([rows, dim], the first is x) and parameters ([dim] fp32) over; the GPU's index."""
    x = tensors[0]
    if not isinstance(x, torch.Tensor):
        _invalid("x: a torch tensor is needed")
    dim, index, dt, tensor, f32 = desc.dim, x.get_device(), _JFA_DTYPE.get(desc.dtype, torch.float32), torch.Tensor, torch.float32
    shape = (desc.rows, dim)
    for i, t in enumerate(tensors):
        if t is not None and not (isinstance(t, tensor) and t.shape == shape and t.dtype is dt
                                  and t.get_device() == index and index >= 0 and t.is_contiguous()):
            _refuse(t, ("x", "block", "gate", "dy", "dn")[i], shape, (dt,), index)
    shape = (dim,)
    for i, t in enumerate(params):
        if t is not None and not (isinstance(t, tensor) and t.shape == shape and t.dtype is f32
                                  and t.get_device() == index and t.is_contiguous()):
            _refuse(t, _BLOCK_NORM_PARAMS[i], shape, (f32,), index)
    return index


def _like(t):
    return None if t is None else torch.empty_like(t)


def block_norm_forward(desc: jfa_block_norm, x, block, gate=None, scale=None, post_gamma=None,
                       post_beta=None, pre_gamma=None, pre_beta=None, stream=None):
    """Allocates and returns (y, n) of jfa_block_norm_forward; n is None
    without a pre_norm."""
    params = (scale, post_gamma, post_beta, pre_gamma, pre_beta)
    s = _stream_here(_block_norm_args(desc, (x, block, gate), params), stream)
    if s is None:
        with _switch(x.device, stream):
            return block_norm_forward(desc, x, block, gate, *params)
    y = torch.empty_like(x)
    n = torch.empty_like(x) if desc.pre_norm else None
    st = (_LIB or load()).jfa_block_norm_forward(
        ctypes.byref(desc), x.data_ptr(), _ptr(block), _ptr(gate), _ptr(scale), _ptr(post_gamma),
        _ptr(post_beta), _ptr(pre_gamma), _ptr(pre_beta), y.data_ptr(), _ptr(n), s)
    if st:
        _check(st)
    return y, n


def block_norm_backward(desc: jfa_block_norm, x, block, gate=None, scale=None, post_gamma=None,
                        post_beta=None, pre_gamma=None, pre_beta=None, dy=None, dn=None, ws=None,
                        stream=None):
    """Allocates and returns the gradients of jfa_block_norm_backward as a dict
    with the keys x, block, gate, scale, post_gamma, post_beta, pre_gamma and
    pre_beta (None for an input that is None)."""
    params = (scale, post_gamma, post_beta, pre_gamma, pre_beta)
    index = _block_norm_args(desc, (x, block, gate, dy, dn), params)
    s = _stream_here(index, stream)
    if s is None:
        with _switch(x.device, stream):
            return block_norm_backward(desc, x, block, gate, *params, dy=dy, dn=dn, ws=ws)
    if ws is None:
        ws = block_norm_workspace(desc, x.device)
    else:
        _buffer(ws, index)
    dx, dblock, dgate = torch.empty_like(x), torch.empty_like(x), _like(gate)
    dscale, dpost_gamma, dpost_beta = _like(scale), _like(post_gamma), _like(post_beta)
    dpre_gamma, dpre_beta = _like(pre_gamma), _like(pre_beta)
    st = (_LIB or load()).jfa_block_norm_backward(
        ctypes.byref(desc), x.data_ptr(), _ptr(block), _ptr(gate), _ptr(scale), _ptr(post_gamma),
        _ptr(post_beta), _ptr(pre_gamma), _ptr(pre_beta), _ptr(dy), _ptr(dn), dx.data_ptr(),
        dblock.data_ptr(), _ptr(dgate), _ptr(dscale), _ptr(dpost_gamma), _ptr(dpost_beta),
        _ptr(dpre_gamma), _ptr(dpre_beta), ws.data_ptr(), ws.numel() * ws.element_size(), s)
    if st:
        _check(st)
    return {"x": dx, "block": dblock, "gate": dgate, "scale": dscale, "post_gamma": dpost_gamma,
            "post_beta": dpost_beta, "pre_gamma": dpre_gamma, "pre_beta": dpre_beta}
