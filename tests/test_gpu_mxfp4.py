"""MXFP4 quantiser, product and linear layer on the GPU against the 64-bit
forms (oracle.mx4).

The quantiser's decisions are integers: codes and scale bytes are compared
for equality.  A product of two E2M1 values and two powers of two is exact in
fp32, so an fp32 result differs from the exact one only by the additions: at
most k + 24 of them (the k terms, up to 8 split ranges, bias and what out
held, with room), each off by at most one unit in the last place (2^-23, which
also covers a sum that truncates) of a partial sum that is bounded by the sum
of the terms' absolute values.  A bf16 result adds half a step, 2^-8 of the
value.
"""
import numpy as np
import pytest
import torch

from jagged_attention_recommender_jfa_b200 import jfa
from oracle import mx4

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def draw(rows, cols, dtype, seed, wide=True):
    """Values over many binades, some zero rows, in the stored dtype."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols))
    if wide:
        x *= np.exp2(rng.integers(-6, 7, size=(rows, 1))) * np.exp2(rng.integers(-4, 5, size=(1, cols)))
        x[rng.random(rows) < 0.1] = 0.0
    return torch.from_numpy(x).to(TORCH[dtype])


def operand_of(x, along_rows=False):
    """The oracle's (codes one per element, scale bytes) of x or its transpose."""
    a = x.double().numpy()
    return mx4.quantize(a.T if along_rows else a)


def check_operand(op, x, along_rows):
    codes, scales = operand_of(x, along_rows)
    assert (op.rows, op.cols) == ((x.shape[1], x.shape[0]) if along_rows else tuple(x.shape))
    assert np.array_equal(mx4.unpack(op.codes.cpu().numpy()), codes)
    assert np.array_equal(op.scales.cpu().numpy(), mx4.tile_scales(scales))
    return mx4.values(codes, scales, op.cols)


SIZES = [(1, 1), (1, 32), (3, 31), (5, 33), (7, 128), (33, 64), (64, 127), (127, 129), (129, 200), (130, 1003),
         (257, 1000), (1, 4097), (300, 8)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("along_rows", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantise_matches_oracle(cuda_device, rows, cols, along_rows, dtype):
    x = draw(rows, cols, dtype, rows * 7 + cols)
    op, deq = jfa.quantize_mxfp4(x.to(cuda_device), along_rows, want_dequant=True)
    v = check_operand(op, x, along_rows)
    assert np.array_equal(deq.double().cpu().numpy(), v.T if along_rows else v)
    plain = jfa.quantize_mxfp4(x.to(cuda_device), along_rows)
    assert torch.equal(plain.codes, op.codes) and torch.equal(plain.scales, op.scales)


@pytest.mark.parametrize("rows,cols", SIZES + [(128, 128), (1000, 520)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantise_both_ways_in_one_pass(cuda_device, rows, cols, dtype):
    x = draw(rows, cols, dtype, rows * 5 + cols)
    x[0, 0] = float("nan")   # one bad block each way
    op, op_t = jfa.quantize_mxfp4_both(x.to(cuda_device))
    check_operand(op, x, False)
    check_operand(op_t, x, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 140])
def test_quantise_both_ways_every_width(cuda_device, dtype, rows):
    for cols in list(range(1, 20)) + list(range(121, 138)) + [257, 1003]:
        x = draw(rows, cols, dtype, cols)
        x[rows // 2, cols // 3] = float("inf")
        op, op_t = jfa.quantize_mxfp4_both(x.to(cuda_device))
        check_operand(op, x, False)
        check_operand(op_t, x, True)


@pytest.mark.parametrize("along_rows", [False, True])
@pytest.mark.parametrize("cols", [256, 131])
def test_quantise_special_values(cuda_device, along_rows, cols):
    # infinities, NaN, the largest and smallest numbers, subnormals, zeros of
    # both signs, rounding ties; each in blocks of its own and mixed
    rng = np.random.default_rng(5)
    x = rng.normal(size=(96, cols)).astype(np.float32)
    x[3, 5] = np.inf
    x[40, 40] = -np.inf
    x[41, 100] = np.nan
    x[64:] *= np.float32(2.0 ** -130)
    x[70, 64] = np.float32(2.0 ** -149)
    x[8, :32] = -0.0
    x[9, :32] = np.float32(3.4e38)
    x[10, :32] = np.array([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 4, np.float32) * 2.0 ** 9
    x[11, :32] = np.finfo(np.float32).tiny
    t = torch.from_numpy(x)
    op, deq = jfa.quantize_mxfp4(t.to(cuda_device), along_rows, want_dequant=True)
    v = check_operand(op, t, along_rows)
    d = deq.double().cpu().numpy()
    assert np.array_equal(d.T if along_rows else d, v, equal_nan=True)
    b = t.to(torch.bfloat16)
    op, deq = jfa.quantize_mxfp4(b.to(cuda_device), along_rows, want_dequant=True)
    v = check_operand(op, b, along_rows)
    d = deq.double().cpu().numpy()
    assert np.array_equal(d.T if along_rows else d, v, equal_nan=True)


@pytest.mark.parametrize("along_rows", [0, 1])
@pytest.mark.parametrize("rows,cols", [(70, 100), (70, 104), (1, 33)])
def test_quantise_writes_its_buffers_and_nothing_else(cuda_device, along_rows, rows, cols):
    x = draw(rows, cols, "bf16", 3)
    r, c = (cols, rows) if along_rows else (rows, cols)
    nc, ns, pad = jfa.jfa_mxfp4_code_bytes(r, c), jfa.jfa_mxfp4_scale_bytes(r, c), 256
    codes = torch.full((nc + pad,), 0xAA, dtype=torch.uint8, device=cuda_device)
    scales = torch.full((ns + pad,), 0xFF, dtype=torch.uint8, device=cuda_device)
    deq = torch.full((rows * cols + pad,), 7.0, dtype=torch.bfloat16, device=cuda_device)
    jfa.jfa_quantize_mxfp4_dequant(x.to(cuda_device), "bf16", rows, cols, along_rows, codes, scales, deq)
    op = jfa.MxOperand(codes[:nc].reshape(r, -1), scales[:ns], r, c)
    check_operand(op, x, along_rows)
    assert (codes[nc:] == 0xAA).all() and (scales[ns:] == 0xFF).all() and (deq[rows * cols:] == 7.0).all()


def product_bound(A, B, k, extra):
    S = np.abs(A) @ np.abs(B).T + extra
    return (k + 24) * 2.0 ** -23 * S


def run_product(dev, m, n, k, out_dtype, bias=False, accumulate=False, seed=0, ws=None):
    x, w = draw(m, k, "bf16", seed + 1), draw(n, k, "bf16", seed + 2)
    A, B = (mx4.values(*operand_of(t), k) for t in (x, w))
    rng = np.random.default_rng(seed + 3)
    b = torch.from_numpy(rng.normal(size=n).astype(np.float32)) if bias else None
    c = torch.from_numpy(rng.normal(size=(m, n))).to(out_dtype) if accumulate else None
    a_op, b_op = jfa.quantize_mxfp4(x.to(dev)), jfa.quantize_mxfp4(w.to(dev))
    out = jfa.matmul_mxfp4(a_op, b_op, bias=None if b is None else b.to(dev), out=None if c is None else c.to(dev),
                           out_dtype=out_dtype, accumulate=accumulate, ws=ws)
    ref = A @ B.T
    extra = np.zeros((m, n))
    if bias:
        ref = ref + b.double().numpy()
        extra = extra + np.abs(b.double().numpy())
    if accumulate:
        ref = ref + c.double().numpy()
        extra = extra + np.abs(c.double().numpy())
    bound = product_bound(A, B, k, extra)
    if out_dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    got = out.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all()
    worst = np.argmax(np.abs(got - ref) - bound)
    assert (np.abs(got - ref) <= bound).all(), (m, n, k, np.unravel_index(worst, got.shape), got.flat[worst], ref.flat[worst])
    return out


PRODUCTS = [(1, 1, 1), (1, 8, 32), (1, 64, 64), (2, 100, 96), (128, 128, 128), (128, 64, 256), (5, 4096, 1024),
            (1, 4096, 4100), (129, 130, 131), (200, 333, 544), (256, 512, 288), (300, 1032, 2008), (77, 65, 8192),
            (1000, 1000, 100), (4099, 257, 513), (64, 64, 160), (65, 191, 224)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_product_matches_oracle(cuda_device, m, n, k, out_dtype):
    run_product(cuda_device, m, n, k, out_dtype, seed=m + n + k)


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (33, 70, 100), (7, 4096, 2048), (300, 260, 700), (2500, 1028, 257)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bias,accumulate", [(True, False), (False, True), (True, True)])
def test_product_epilogue(cuda_device, m, n, k, out_dtype, bias, accumulate):
    run_product(cuda_device, m, n, k, out_dtype, bias, accumulate, seed=m * 3 + k)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_empty_sum(cuda_device, out_dtype):
    dev = cuda_device
    a = jfa.quantize_mxfp4(torch.zeros(150, 0, device=dev))
    b = jfa.quantize_mxfp4(torch.zeros(70, 0, device=dev))
    bias = torch.arange(70, dtype=torch.float32, device=dev)
    assert torch.equal(jfa.matmul_mxfp4(a, b, out_dtype=out_dtype), torch.zeros(150, 70, dtype=out_dtype, device=dev))
    got = jfa.matmul_mxfp4(a, b, bias=bias, out=torch.ones(150, 70, dtype=out_dtype, device=dev), accumulate=True)
    assert torch.equal(got, (bias + 1).to(out_dtype).expand(150, 70))
    none = jfa.matmul_mxfp4(jfa.quantize_mxfp4(torch.zeros(0, 64, device=dev)),
                            jfa.quantize_mxfp4(torch.zeros(70, 64, device=dev)))
    assert none.shape == (0, 70)


@pytest.mark.parametrize("m,n,k,row,col", [(3, 70, 256, 1, 200), (300, 300, 1000, 131, 999), (1, 4096, 2048, 0, 2000)])
def test_nan_blocks_reach_their_row_only(cuda_device, m, n, k, row, col):
    x, w = draw(m, k, "bf16", 1, wide=False), draw(n, k, "bf16", 2, wide=False)
    x[row, col] = float("inf")
    out = jfa.matmul_mxfp4(jfa.quantize_mxfp4(x.to(cuda_device)), jfa.quantize_mxfp4(w.to(cuda_device)),
                           out_dtype=torch.float32)
    bad = torch.isnan(out).cpu()
    assert bad[row].all() and bad.sum() == n


def test_product_exact_small_integers(cuda_device):
    # every product and sum is a small multiple of a power of two: no rounding
    # at all, so a wrong operand, scale or K step shows as a difference
    rng = np.random.default_rng(9)
    m, n, k = 200, 264, 704
    a = rng.integers(-3, 4, (m, k)).astype(np.float32) * np.exp2(rng.integers(-2, 3, (m, k // 32))).repeat(32, 1)
    b = rng.integers(-3, 4, (n, k)).astype(np.float32) * np.exp2(rng.integers(-2, 3, (n, k // 32))).repeat(32, 1)
    a[:, ::32] = 6 * np.exp2(rng.integers(-2, 3, (m, k // 32)))   # fixes each block's exponent
    b[:, ::32] = 6 * np.exp2(rng.integers(-2, 3, (n, k // 32)))
    a, b = a.astype(np.float32), b.astype(np.float32)
    A, B = (mx4.values(*mx4.quantize(t), k) for t in (a, b))
    out = jfa.matmul_mxfp4(*(jfa.quantize_mxfp4(torch.from_numpy(t).to(cuda_device)) for t in (a, b)),
                           out_dtype=torch.float32)
    ref = A @ B.T
    assert np.abs(ref).max() < 2.0 ** 20 and np.array_equal(ref * 2.0 ** 4, np.round(ref * 2.0 ** 4))
    assert np.array_equal(out.double().cpu().numpy(), ref)


def test_product_leaves_what_lies_behind_the_result(cuda_device):
    for m, n, k in ((130, 100, 96), (3, 33, 64), (1, 8, 4096)):
        x, w = draw(m, k, "bf16", 1).to(cuda_device), draw(n, k, "bf16", 2).to(cuda_device)
        a, b = jfa.quantize_mxfp4(x), jfa.quantize_mxfp4(w)
        ref = jfa.matmul_mxfp4(a, b)
        buf = torch.full((m * n + 512,), 7.0, dtype=torch.bfloat16, device=cuda_device)
        jfa.jfa_matmul_mxfp4(m, n, k, a.codes, a.scales, b.codes, b.scales, None, buf, "bf16", 0,
                             jfa.mxfp4_workspace(cuda_device))
        assert torch.equal(buf[:m * n].reshape(m, n), ref) and (buf[m * n:] == 7.0).all()


def test_product_repeats_bit_for_bit(cuda_device):
    ws = jfa.mxfp4_workspace(cuda_device)
    for m, n, k in ((1, 4096, 4096), (700, 900, 2080)):
        first = run_product(cuda_device, m, n, k, torch.float32, seed=4, ws=ws)
        for _ in range(3):
            assert torch.equal(run_product(cuda_device, m, n, k, torch.float32, seed=4, ws=ws), first)
    jfa.jfa_check_error(ws)


def linear_reference(x, w, dy):
    """x, w, dy fp64 arrays -> y, dx, dw and the sums of absolute terms of each."""
    q = lambda t: mx4.values(*mx4.quantize(t), t.shape[1])
    pairs = {"y": (q(x), q(w)), "dx": (q(dy), q(w.T)), "dw": (q(dy.T), q(x.T))}
    return {n: (a @ b.T, np.abs(a) @ np.abs(b).T, a.shape[1]) for n, (a, b) in pairs.items()}


@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (5, 128, 96), (333, 200, 131), (1025, 260, 516)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_forward_and_backward(cuda_device, m, n, k, dtype):
    x, w, dy = draw(m, k, dtype, 1), draw(n, k, dtype, 2), draw(m, n, dtype, 3)
    ref = linear_reference(*(t.double().numpy() for t in (x, w, dy)))
    X, W, DY = (t.to(cuda_device) for t in (x, w, dy))
    y = jfa.linear_mxfp4_forward(X, jfa.quantize_mxfp4(W))
    dx, dw = jfa.linear_mxfp4_backward(DY, X, jfa.quantize_mxfp4(W, along_rows=True))
    _, dw2 = jfa.linear_mxfp4_backward(DY, X, jfa.quantize_mxfp4(W, along_rows=True), dw=dw.clone())
    assert dx.dtype == y.dtype == TORCH[dtype] and dw.dtype == torch.float32
    for name, got in (("y", y), ("dx", dx), ("dw", dw), ("dw2", dw2)):
        r, S, terms = ref["dw" if name == "dw2" else name]
        if name == "dw2":
            r, S = 2 * r, 2 * S
        bound = (terms + 24) * 2.0 ** -23 * S
        if got.dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * (np.abs(r) + bound)
        assert (np.abs(got.double().cpu().numpy() - r) <= bound).all(), name


@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (37, 66, 131), (300, 257, 100), (5, 0, 40), (5, 40, 0), (0, 40, 33)])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_linear_entries_equal_their_parts(cuda_device, m, n, k, accumulate):
    # the one-call passes write what the quantiser and the product write, and
    # nothing behind their buffers
    dev, pad = cuda_device, 64
    x, w, dy = (draw(*s, "bf16", i).to(dev) for i, s in enumerate([(m, k), (n, k), (m, n)]))
    bias = torch.randn(n, generator=torch.Generator().manual_seed(1)).to(dev)
    wq, wt, ws = jfa.quantize_mxfp4(w), jfa.quantize_mxfp4(w, along_rows=True), jfa.mxfp4_workspace(dev)

    def guarded(count, dtype, value):
        return torch.full((count + pad,), value, dtype=dtype, device=dev)

    def left_alone(*pairs):
        return all((t[count:] == value).all() for t, count, value in pairs)

    ny, nx, nw = m * n, m * k, n * k
    sizes = [jfa.jfa_linear_mxfp4_scratch_bytes(m, n, k, b) for b in (0, 1)]
    s0, s1 = (guarded(c, torch.uint8, 0xEE) for c in sizes)
    y, dx = guarded(ny, torch.bfloat16, 7.0), guarded(nx, torch.bfloat16, 7.0)
    dw = guarded(nw, torch.float32, 0.5)
    jfa.jfa_linear_mxfp4_forward(x, "bf16", m, n, k, wq.codes, wq.scales, bias, y, s0, ws, scratch_bytes=sizes[0])
    jfa.jfa_linear_mxfp4_backward(dy, "bf16", x, "bf16", m, n, k, wt.codes, wt.scales, dx, dw, accumulate, s1, ws,
                                  scratch_bytes=sizes[1])
    jfa.jfa_check_error(ws)
    assert left_alone((s0, sizes[0], 0xEE), (s1, sizes[1], 0xEE), (y, ny, 7.0), (dx, nx, 7.0), (dw, nw, 0.5))
    g, gt, xt = jfa.quantize_mxfp4(dy), jfa.quantize_mxfp4(dy, True), jfa.quantize_mxfp4(x, True)
    held = torch.full((n, k), 0.5, device=dev)
    assert torch.equal(y[:ny].view(m, n), jfa.matmul_mxfp4(jfa.quantize_mxfp4(x), wq, bias))
    assert torch.equal(dx[:nx].view(m, k), jfa.matmul_mxfp4(g, wt))
    assert torch.equal(dw[:nw].view(n, k), jfa.matmul_mxfp4(gt, xt, out=held, accumulate=bool(accumulate)))


def test_linear_of_no_tokens(cuda_device):
    x, dy = (torch.zeros(0, c, dtype=torch.bfloat16, device=cuda_device) for c in (64, 96))
    w = draw(96, 64, "bf16", 1).to(cuda_device)
    assert jfa.linear_mxfp4_forward(x, jfa.quantize_mxfp4(w)).shape == (0, 96)
    dx, dw = jfa.linear_mxfp4_backward(dy, x, jfa.quantize_mxfp4(w, along_rows=True))
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(96, 64, device=cuda_device))


def test_streams_and_graph_capture(cuda_device):
    # two streams at once share an error word; a captured linear layer replays
    # on new data written into its inputs
    dev = cuda_device
    ws = jfa.mxfp4_workspace(dev)
    xs = [draw(300, 520, "bf16", s).to(dev) for s in range(4)]
    w = jfa.quantize_mxfp4(draw(200, 520, "bf16", 9).to(dev))
    want = [jfa.linear_mxfp4_forward(x, w, ws=ws) for x in xs]
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    torch.cuda.synchronize()
    got = [jfa.linear_mxfp4_forward(x, w, ws=ws, stream=streams[i % 2], check=False) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = jfa.linear_mxfp4_forward(x, w, ws=ws, check=False)
    for src, ref in zip(xs, want):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
    jfa.jfa_check_error(ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 136, 300])
def test_quantise_every_place_of_a_row_in_its_vectors(cuda_device, dtype, rows):
    # narrow rows (several in a vector), rows that end anywhere around a column
    # tile, with bad blocks beside good ones; a guard behind every buffer
    rng = np.random.default_rng(rows)
    for cols in list(range(1, 42)) + list(range(121, 138)) + [255, 257, 1003]:
        x = draw(rows, cols, dtype, cols)
        x[torch.from_numpy(rng.random((rows, cols)) < 0.004)] = float("nan")
        x[torch.from_numpy(rng.random((rows, cols)) < 0.002)] = -float("inf")
        x[rows // 2] *= 2.0 ** -120
        nc, ns, n, pad = jfa.jfa_mxfp4_code_bytes(rows, cols), jfa.jfa_mxfp4_scale_bytes(rows, cols), rows * cols, 64
        for deq in (torch.full((n + pad,), 7.0, dtype=TORCH[dtype], device=cuda_device), None):
            codes = torch.full((nc + pad,), 0xAA, dtype=torch.uint8, device=cuda_device)
            scales = torch.full((ns + pad,), 0xEE, dtype=torch.uint8, device=cuda_device)
            if deq is None:
                jfa.jfa_quantize_mxfp4(x.to(cuda_device), dtype, rows, cols, 0, codes, scales)
            else:
                jfa.jfa_quantize_mxfp4_dequant(x.to(cuda_device), dtype, rows, cols, 0, codes, scales, deq)
            v = check_operand(jfa.MxOperand(codes[:nc].reshape(rows, -1), scales[:ns], rows, cols), x, False)
            assert (codes[nc:] == 0xAA).all() and (scales[ns:] == 0xEE).all()
            if deq is not None:
                got = deq[:n].reshape(rows, cols).double().cpu().numpy()
                assert np.array_equal(got, v, equal_nan=True), cols
                assert np.array_equal(np.signbit(got) & ~np.isnan(v), np.signbit(v) & ~np.isnan(v)), cols
                assert (deq[n:] == 7.0).all()


@pytest.mark.parametrize("along_rows", [False, True])
def test_quantise_offsets_past_32_bits(cuda_device, along_rows):
    # 2.2e9 elements: the last rows (of whole scale tiles) against the same rows alone
    rows, cols = 2_240_000, 1000
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=cuda_device)
    x[-128:] = torch.randn(128, cols, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(cuda_device)
    assert rows % 128 == 0 and rows * cols > 1 << 31
    op, deq = jfa.quantize_mxfp4(x, along_rows, want_dequant=True)
    alone, d = jfa.quantize_mxfp4(x[-128:].clone(), along_rows, want_dequant=True)
    assert torch.equal(deq[-128:], d) and (deq[:-128] == 0).all()
    if along_rows:
        assert torch.equal(op.codes[:, -64:], alone.codes)
        at = op.scales.view(8, rows // 128, 512)
        assert torch.equal(at[:, -1].reshape(-1), alone.scales)
    else:
        assert torch.equal(op.codes[-128:], alone.codes)
        assert torch.equal(op.scales[-alone.scales.numel():], alone.scales)


def test_quantise_offsets_past_32_bits_off_boundaries(cuda_device):
    rows, cols = 2_240_008, 999
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=cuda_device)
    x[-136:] = draw(136, cols, "bf16", 1).to(cuda_device)
    op, deq = jfa.quantize_mxfp4(x, want_dequant=True)
    alone, d = jfa.quantize_mxfp4(x[-136:].clone(), want_dequant=True)
    assert rows % 128 == 8 and rows * cols > 1 << 31
    assert torch.equal(deq[-136:], d) and (deq[:-136] == 0).all()
    assert torch.equal(op.codes[-136:], alone.codes)
    assert torch.equal(op.scales[-alone.scales.numel():], alone.scales)


def test_product_offsets_past_32_bits(cuda_device):
    # 2.3e9 results; the last rows against the same rows alone
    m, n, k = 560_128, 4096, 64
    x = draw(256, k, "bf16", 1).to(cuda_device)
    w = jfa.quantize_mxfp4(draw(n, k, "bf16", 2).to(cuda_device))
    big = torch.zeros(m, k, dtype=torch.bfloat16, device=cuda_device)
    big[-256:] = x
    ref = jfa.matmul_mxfp4(jfa.quantize_mxfp4(x), w)
    out = jfa.matmul_mxfp4(jfa.quantize_mxfp4(big), w)
    assert torch.equal(out[-256:], ref) and (out[:-256] == 0).all()
    odd = torch.zeros(m, 4097, dtype=torch.bfloat16, device=cuda_device)   # rows off every boundary
    w1 = jfa.quantize_mxfp4(torch.cat([draw(n, k, "bf16", 2), draw(1, k, "bf16", 3)]).to(cuda_device))
    jfa.matmul_mxfp4(jfa.quantize_mxfp4(big), w1, out=odd)
    assert torch.equal(odd[-256:, :4096], ref) and (odd[:-256] == 0).all()


# one CTA per tile, a split contraction over a cluster, a pair of CTAs (one
# stage, and more than its ring holds)
@pytest.mark.parametrize("m,n,k", [(100, 8192, 256), (64, 64, 8192), (300, 512, 256), (300, 512, 8192)])
def test_bounded_waits_end_in_an_error(cuda_device, m, n, k):
    # a load that never comes: the waits give up, the call reports it, and the
    # same workspace and buffers work again
    ws = jfa.mxfp4_workspace(cuda_device)
    a, b = (jfa.quantize_mxfp4(draw(r, k, "bf16", r).to(cuda_device)) for r in (m, n))
    want = jfa.matmul_mxfp4(a, b, ws=ws)
    out = torch.empty_like(want)
    jfa.jfa_test_inject(jfa.JFA_TEST_MATMUL_SKIP_LOAD)
    with pytest.raises(jfa.JfaError) as ei:
        jfa.matmul_mxfp4(a, b, out=out, ws=ws)
    assert ei.value.status == jfa.JFA_ERR_TIMEOUT
    assert torch.equal(jfa.matmul_mxfp4(a, b, out=out, ws=ws), want)
