"""Cases of the operators around the attention of a block: the MXFP4
quantiser, the MXFP4 product and the linear layer built on it, and the norms
before and after a block fused with its gate and residual scale.

Formats (OCP MX v1.0, E2M1 elements, one E8M0 scale per 32).  An operand of R
rows and K columns is held as
  codes  : uint8 [R][Kp / 2], Kp = K rounded up to 32, element 2i in the low
           four bits of byte i, zero codes behind column K
  scales : uint8, 128 x 4 tiles: the byte of (row r, block c) is at
           ((r / 128) * T + c / 4) * 512 + (r % 32) * 16 + (r / 32 % 4) * 4 + c % 4
           with T = ceil(Kp / 128), zero behind the last row and block.

``own`` is set by the tool that imports this file: false runs the plain forms
(elementary torch operations in 32 bits), true the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def _quant(rows, cols, along_rows, dtype, name=None):
    c = dict(op="quantize", rows=rows, cols=cols, along_rows=along_rows, dtype=dtype)
    return dict(c, name=name) if name else c


def _prod(m, n, k, out, bias, name=None):
    c = dict(op="product", m=m, n=n, k=k, out=out, bias=bias)
    return dict(c, name=name) if name else c


def _lin(op, m, n, k, name=None):
    c = dict(op=op, m=m, n=n, k=k)
    return dict(c, name=name) if name else c


def _norm(op, rows, dim, dtype, post, pre, gate, scale, name=None):
    c = dict(op=op, rows=rows, dim=dim, dtype=dtype, post=post, pre=pre, gate=gate, scale=scale)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the tokens of a few users' last events, quantised before a projection
        _quant(7, 1024, False, "bf16", "quant_tokens"),
        # every token of the 256-sequence training batch at model width 8 x 128
        _quant(222283, 1024, False, "bf16", "quant_batch"),
        # a weight gradient's operand: blocks run along the tokens, odd sizes, fp32
        _quant(20011, 1000, True, "f32", "quant_cols_odd"),
        # one token through a projection: latency
        _prod(1, 4096, 1024, "bf16", False, "product_token"),
        # ragged sizes, fp32 result with a bias
        _prod(4999, 1032, 2008, "f32", True, "product_ragged"),
        # a wide layer over a long batch
        _prod(32768, 4096, 4096, "bf16", False, "product_large"),
        # the four projections of a gated attention block in one, over the training batch
        _lin("linear_fwd", 222283, 4096, 1024, "linear_fwd"),
        # the same layer's gradients for an odd number of tokens
        _lin("linear_bwd", 65537, 4096, 1024, "linear_bwd"),
        # a handful of tokens between two blocks: latency
        _norm("norm_fwd", 4, 1024, "bf16", "rms", "rms", "silu", True, "norm_fwd_tokens"),
        # the training batch between two blocks, both directions
        _norm("norm_fwd", 222283, 1024, "bf16", "rms", "rms", "silu", True, "norm_fwd_batch"),
        _norm("norm_bwd", 222283, 1024, "bf16", "rms", "rms", "silu", True, "norm_bwd_batch"),
        # LayerNorms of a width that is no multiple of a vector, in fp32
        _norm("norm_bwd", 9001, 1003, "f32", "layer", "layer", "sigmoid", True, "norm_bwd_odd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the logarithm of the listed ranges."""
    op = rng.choice(("quantize", "product", "linear_fwd", "linear_bwd", "norm_fwd", "norm_bwd"))
    if op == "quantize":
        cols = _log(rng, 32, 8192)
        rows = _log(rng, 1, min(262144, (1 << 27) // cols))
        return _quant(rows, cols, rng.random() < 0.5, rng.choice(("bf16", "f32")))
    if op == "product":
        n, k = _log(rng, 8, 8192), _log(rng, 32, 8192)
        m = _log(rng, 1, max(2, min(131072, (1 << 38) // (n * k))))
        return _prod(m, n, k, rng.choice(("bf16", "f32")), rng.random() < 0.5)
    if op in ("linear_fwd", "linear_bwd"):
        n, k = _log(rng, 64, 4096), _log(rng, 64, 4096)
        m = _log(rng, 1, min(131072, (1 << 37) // (n * k)))
        return _lin(op, m, n, k)
    dim = _log(rng, 32, 8192)
    rows = _log(rng, 1, min(131072, (1 << 26) // dim))
    return _norm(op, rows, dim, rng.choice(("bf16", "f32")), rng.choice(("none", "rms", "layer")),
                 rng.choice(("none", "rms", "layer")), rng.choice(("none", "identity", "silu", "sigmoid")),
                 rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFFFFFF)


def _activations(rows, cols, dtype, seed, salt):
    """Tokens' activations: unit normals with a few wide channels and some
    all-zero rows (padding tokens)."""
    g = _gen(seed, salt)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    if rows > 16:
        x[torch.randint(0, rows, (rows // 64 + 1,), generator=g, device=DEV)] = 0.0
    return x.to(DTYPES[dtype])


def _weights(rows, cols, dtype, seed, salt):
    g = _gen(seed, salt)
    return (torch.randn(rows, cols, generator=g, device=DEV) / math.sqrt(cols)).to(DTYPES[dtype])


def _up(a, b):
    return (a + b - 1) // b * b


def _exponents(blocks):
    """Shared exponents of fp32 blocks [..., 32]."""
    amax = blocks.abs().amax(-1)
    _, e = torch.frexp(amax)
    x = (e - 3).clamp(-127, 127)
    return torch.where(amax == 0, torch.full_like(x, -127), x)


def _indexes(mag):
    """Round-to-nearest-even index into E2M1 of magnitudes (saturating)."""
    return ((mag > 0.25).to(torch.uint8) + (mag >= 0.75) + (mag > 1.25) + (mag >= 1.75)
            + (mag > 2.5) + (mag >= 3.5) + (mag > 5.0))


def _quantize_plain(x):
    """x [R, K] -> (signed values on the E2M1 grid before scaling as [R, Kp/32, 32]
    indexes and signs, exponents [R, Kp/32])."""
    rows, k = x.shape
    kp = _up(k, 32)
    f = x.float()
    if kp != k:
        f = torch.nn.functional.pad(f, (0, kp - k))
    f = f.reshape(rows, kp // 32, 32)
    ex = _exponents(f)
    scaled = torch.ldexp(f, -ex.unsqueeze(-1))
    return _indexes(scaled.abs()), torch.signbit(f), ex


def _values_plain(x):
    rows, k = x.shape
    idx, neg, ex = _quantize_plain(x)
    table = torch.tensor(E2M1, device=x.device)
    v = torch.ldexp(table[idx.long()], ex.unsqueeze(-1))
    return torch.where(neg, -v, v).reshape(rows, -1)[:, :k]


def _tile_scales(s):
    """[R, Kp/32] bytes -> the tiled layout."""
    r, c = s.shape
    rt, kt = _up(r, 128) // 128, _up(c, 4) // 4
    full = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8, device=s.device)
    full[:r, :c] = s
    return full.reshape(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def _untile_scales(s, rows, blocks):
    rt, kt = _up(rows, 128) // 128, _up(blocks, 4) // 4
    return s.reshape(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :blocks]


def _operand(x):
    """(codes, scales) of x [R, K], as a producer leaves them."""
    rows = x.shape[0]
    idx, neg, ex = _quantize_plain(x)
    code = (idx | (neg.to(torch.uint8) << 3)).reshape(rows, -1)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), _tile_scales((ex + 127).to(torch.uint8))


def _decode(codes, scales, rows, k):
    """Values (fp32) of an operand."""
    both = torch.stack((codes & 15, codes >> 4), -1).reshape(rows, -1)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    ex = _untile_scales(scales, rows, both.shape[1] // 32).int() - 127
    v = torch.ldexp(table[both.long()].reshape(rows, -1, 32), ex.unsqueeze(-1))
    return v.reshape(rows, -1)[:, :k]


def prepare(case, seed):
    op = case["op"]
    st = dict(case=case)
    if op == "quantize":
        st["x"] = _activations(case["rows"], case["cols"], case["dtype"], seed, 1)
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"] = _operand(_activations(m, k, "bf16", seed, 1))
        st["b"] = _operand(_weights(n, k, "bf16", seed, 2))
        if case["bias"]:
            st["bias"] = torch.randn(n, generator=_gen(seed, 3), device=DEV)
    elif op == "linear_fwd":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"] = _activations(m, k, "bf16", seed, 1)
        st["w"] = _operand(_weights(n, k, "bf16", seed, 2))
        st["bias"] = torch.randn(n, generator=_gen(seed, 3), device=DEV)
    elif op == "linear_bwd":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"] = _activations(m, k, "bf16", seed, 1)
        st["w"] = _weights(n, k, "bf16", seed, 2)
        st["dy"] = _activations(m, n, "bf16", seed, 3)
    else:
        st.update(_norm_inputs(case, seed))
    if own:
        from jagged_attention_recommender_jfa_b200 import jfa
        if op in ("product", "linear_fwd", "linear_bwd"):
            st["ws"] = jfa.mxfp4_workspace(torch.device(DEV))
        if op in ("norm_fwd", "norm_bwd"):
            st["desc"] = jfa.make_block_norm(rows=case["rows"], dim=case["dim"], dtype=case["dtype"],
                                             post_norm=case["post"], pre_norm=case["pre"], gate=case["gate"])
        if op == "norm_bwd":
            st["ws"] = jfa.block_norm_workspace(st["desc"], torch.device(DEV))
    return st


def _norm_inputs(case, seed):
    rows, dim, dt = case["rows"], case["dim"], case["dtype"]
    st = dict(x=_activations(rows, dim, dt, seed, 1), block=_activations(rows, dim, dt, seed, 2))
    st["gate"] = _activations(rows, dim, dt, seed, 3) if case["gate"] != "none" else None
    g = _gen(seed, 4)
    near_one = lambda: 1.0 + 0.2 * torch.randn(dim, generator=g, device=DEV)
    small = lambda: 0.1 * torch.randn(dim, generator=g, device=DEV)
    st["scale"] = 0.5 * near_one() if case["scale"] else None
    st["post_gamma"] = near_one() if case["post"] != "none" else None
    st["post_beta"] = small() if case["post"] == "layer" else None
    st["pre_gamma"] = near_one() if case["pre"] != "none" else None
    st["pre_beta"] = small() if case["pre"] == "layer" else None
    if case["op"] == "norm_bwd":
        st["dy"] = torch.randn(rows, dim, generator=g, device=DEV).to(DTYPES[dt])
        st["dn"] = torch.randn(rows, dim, generator=g, device=DEV).to(DTYPES[dt]) if case["pre"] != "none" else None
    return st


# ---------------------------------------------------------------------------
# plain forms and the framework's calls
# ---------------------------------------------------------------------------

EPS = 1e-5
PARAMS = ("scale", "post_gamma", "post_beta", "pre_gamma", "pre_beta")


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        x = st["x"]
        v = _values_plain(x.t()).t() if case["along_rows"] else _values_plain(x)
        return v.to(x.dtype).contiguous()
    if op == "product":
        out = _decode(*st["a"], case["m"], case["k"]) @ _decode(*st["b"], case["n"], case["k"]).t()
        if case["bias"]:
            out = out + st["bias"]
        return out.to(DTYPES[case["out"]])
    if op == "linear_fwd":
        out = _values_plain(st["x"]) @ _decode(*st["w"], case["n"], case["k"]).t() + st["bias"]
        return out.to(torch.bfloat16)
    if op == "linear_bwd":
        dx = _values_plain(st["dy"]) @ _values_plain(st["w"].t()).t()
        dw = _values_plain(st["dy"].t()) @ _values_plain(st["x"].t()).t()
        return dx.to(torch.bfloat16), dw
    return _norm_plain(st)


def _stats(v, kind):
    """(centred v, 1 / its root mean square)."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    return v, 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def _norm_plain(st):
    case = st["case"]
    dt = DTYPES[case["dtype"]]
    x, b = st["x"].float(), st["block"].float()
    if case["post"] == "none":
        hat, p = None, b
    else:
        c, r = _stats(b, case["post"])
        hat = c * r
        p = hat * st["post_gamma"]
        if st["post_beta"] is not None:
            p = p + st["post_beta"]
    if case["gate"] == "none":
        a = torch.ones((), device=x.device)
    else:
        u = st["gate"].float()
        sg = 1.0 / (1.0 + torch.exp(-u))
        a = {"identity": u, "silu": u * sg, "sigmoid": sg}[case["gate"]]
    s = st["scale"] if case["scale"] else torch.ones((), device=x.device)
    y = x + s * a * p
    if case["pre"] != "none":
        yc, yr = _stats(y, case["pre"])
        yhat = yc * yr
    if case["op"] == "norm_fwd":
        if case["pre"] == "none":
            return y.to(dt)
        n = yhat * st["pre_gamma"]
        if st["pre_beta"] is not None:
            n = n + st["pre_beta"]
        return y.to(dt), n.to(dt)

    def through(hat, r, g, kind):
        t = g - hat * (g * hat).mean(-1, keepdim=True)
        if kind == "layer":
            t = t - g.mean(-1, keepdim=True)
        return t * r

    grads = {}
    d = st["dy"].float()
    if case["pre"] != "none":
        dn = st["dn"].float()
        grads["pre_gamma"] = (dn * yhat).sum(0)
        if st["pre_beta"] is not None:
            grads["pre_beta"] = dn.sum(0)
        d = d + through(yhat, yr, dn * st["pre_gamma"], case["pre"])
    out = [d.to(dt)]
    if case["scale"]:
        grads["scale"] = (d * a * p).sum(0)
    dp = d * s * a
    if case["post"] == "none":
        out.append(dp.to(dt))
    else:
        grads["post_gamma"] = (dp * hat).sum(0)
        if st["post_beta"] is not None:
            grads["post_beta"] = dp.sum(0)
        out.append(through(hat, r, dp * st["post_gamma"], case["post"]).to(dt))
    if case["gate"] != "none":
        da = d * s * p
        du = {"identity": da, "silu": da * sg * (1.0 + u * (1.0 - sg)),
              "sigmoid": da * sg * (1.0 - sg)}[case["gate"]]
        out.append(du.to(dt))
    return out + [grads[k] for k in PARAMS if k in grads]


def _run_own(st):
    from jagged_attention_recommender_jfa_b200 import jfa
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        return jfa.quantize_mxfp4(st["x"], along_rows=case["along_rows"], want_dequant=True)[1]
    if op == "product":
        a = jfa.MxOperand(*st["a"], case["m"], case["k"])
        b = jfa.MxOperand(*st["b"], case["n"], case["k"])
        return jfa.matmul_mxfp4(a, b, bias=st.get("bias"), out_dtype=DTYPES[case["out"]], ws=st["ws"],
                                check=False)
    if op == "linear_fwd":
        w = jfa.MxOperand(*st["w"], case["n"], case["k"])
        return jfa.linear_mxfp4_forward(st["x"], w, bias=st["bias"], ws=st["ws"], check=False)
    if op == "linear_bwd":
        wt = jfa.quantize_mxfp4(st["w"], along_rows=True)
        return jfa.linear_mxfp4_backward(st["dy"], st["x"], wt, ws=st["ws"], check=False)
    kw = {k: st[k] for k in ("gate",) + PARAMS}
    if op == "norm_fwd":
        y, n = jfa.block_norm_forward(st["desc"], st["x"], st["block"], **kw)
        return y if n is None else (y, n)
    g = jfa.block_norm_backward(st["desc"], st["x"], st["block"], dy=st["dy"], dn=st["dn"], ws=st["ws"], **kw)
    return [g[k] for k in ("x", "block", "gate") + PARAMS if g[k] is not None]


# ---------------------------------------------------------------------------
# work and 64-bit values
# ---------------------------------------------------------------------------


def _operand_bytes(rows, k):
    return rows * (_up(k, 32) // 2 + _up(k, 32) // 32)


def work(case):
    op = case["op"]
    if op == "quantize":
        e = ESIZE[case["dtype"]]
        n = case["rows"] * case["cols"]
        held = _operand_bytes(case["cols"], case["rows"]) if case["along_rows"] else _operand_bytes(case["rows"], case["cols"])
        return {"bytes": 2 * n * e + held, "flops": 4 * n}
    if op in ("product", "linear_fwd", "linear_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "product":
            b = _operand_bytes(m, k) + _operand_bytes(n, k) + m * n * ESIZE[case["out"]] + (4 * n if case["bias"] else 0)
            return {"bytes": b, "flops": 2 * m * n * k}
        if op == "linear_fwd":
            return {"bytes": 2 * m * k + _operand_bytes(n, k) + 2 * m * n + 4 * n, "flops": 2 * m * n * k}
        return {"bytes": 2 * m * n + 2 * m * k + 2 * n * k + 2 * m * k + 4 * n * k, "flops": 4 * m * n * k}
    nel, e = case["rows"] * case["dim"], ESIZE[case["dtype"]]
    gate, pre = case["gate"] != "none", case["pre"] != "none"
    if op == "norm_fwd":
        tensors = 3 + gate + pre
        return {"bytes": nel * e * tensors + 20 * case["dim"], "flops": 16 * nel}
    tensors = 5 + 2 * gate + pre
    return {"bytes": nel * e * tensors + 40 * case["dim"], "flops": 40 * nel}


def _grid_exact(x):
    """E2M1 / E8M0 values of the rows of x, in 64 bits: the nearest point of
    the scaled grid, of two equally near ones the one with the even index."""
    rows, k = x.shape
    out = torch.empty(rows, k, dtype=torch.float64, device=x.device)
    pts = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 25) // max(k, 1))
    for r0 in range(0, rows, step):
        f = x[r0:r0 + step].double()
        pad = torch.zeros(f.shape[0], _up(k, 32) - k, dtype=torch.float64, device=x.device)
        f = torch.cat((f, pad), 1).reshape(-1, 32)
        top = f.abs().max(1, keepdim=True).values
        pw = torch.floor(torch.log2(torch.where(top == 0, torch.ones_like(top), top)))
        pw = torch.where(torch.exp2(pw) > top, pw - 1, pw)       # log2 rounded up to a power of two
        pw = torch.where(torch.exp2(pw + 1) <= top, pw + 1, pw)  # ... or down past one
        unit = torch.exp2((pw - 2).clamp(-127, 127))
        t = (f.abs() / unit).clamp(max=6.0)
        hi = torch.searchsorted(pts, t).clamp(max=7)
        lo = (hi - 1).clamp(min=0)
        dh, dl = (pts[hi] - t).abs(), (t - pts[lo]).abs()
        pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        v = torch.copysign(pts[pick] * unit, f)
        out[r0:r0 + step] = v.reshape(-1, _up(k, 32))[:, :k]
    return out


def _operand_exact(operand, rows, k):
    codes, scales = operand
    c = torch.empty(rows, codes.shape[1] * 2, dtype=torch.int64, device=codes.device)
    c[:, 0::2] = codes.long() % 16
    c[:, 1::2] = codes.long() // 16
    pts = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    v = pts[c % 8] * (1 - 2 * (c // 8)).double()
    r = torch.arange(rows, device=codes.device).unsqueeze(1)
    j = torch.arange(c.shape[1] // 32, device=codes.device).unsqueeze(0)
    tiles = (c.shape[1] + 127) // 128
    at = (r // 128 * tiles + j // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + j % 4
    unit = torch.exp2(scales[at].double() - 127.0)
    return (v * unit.repeat_interleave(32, 1))[:, :k]


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "quantize":
        return _grid_exact(st["x"].t()).t().contiguous() if case["along_rows"] else _grid_exact(st["x"])
    if op == "product":
        out = _operand_exact(st["a"], case["m"], case["k"]) @ _operand_exact(st["b"], case["n"], case["k"]).T
        return out + st["bias"].double() if case["bias"] else out
    if op == "linear_fwd":
        w = _operand_exact(st["w"], case["n"], case["k"])
        return torch.addmm(st["bias"].double(), _grid_exact(st["x"]), w.T)
    if op == "linear_bwd":
        dx = _grid_exact(st["dy"]) @ _grid_exact(st["w"].T.contiguous()).T
        dw = _grid_exact(st["dy"].T.contiguous()) @ _grid_exact(st["x"].T.contiguous()).T
        return dx, dw
    return _norm_exact(case, st)


def _norm_exact(case, st):
    """The formula in 64 bits, over pieces of rows; gradients by torch's
    differentiation of it."""
    back = case["op"] == "norm_bwd"
    par = {k: st[k].double().requires_grad_(back) for k in PARAMS if st[k] is not None}
    step = max(1, (1 << 24) // case["dim"])
    rows_out, sums = None, [torch.zeros_like(p) for p in par.values()]

    def norm(v, kind, which):
        if kind == "none":
            return v
        if kind == "rms":
            return v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * par[which + "_gamma"]
        var, mu = torch.var_mean(v, 1, keepdim=True, correction=0)
        return (v - mu) * torch.rsqrt(var + EPS) * par[which + "_gamma"] + par[which + "_beta"]

    for r0 in range(0, case["rows"], step):
        cut = lambda k: st[k][r0:r0 + step].double()
        x, b = cut("x").requires_grad_(back), cut("block").requires_grad_(back)
        leaves = [x, b]
        t = norm(b, case["post"], "post")
        if case["gate"] != "none":
            u = cut("gate").requires_grad_(back)
            leaves.append(u)
            t = t * {"identity": lambda z: z, "silu": lambda z: z * torch.sigmoid(z), "sigmoid": torch.sigmoid}[case["gate"]](u)
        if case["scale"]:
            t = t * par["scale"]
        y = x + t
        got = [y] if case["pre"] == "none" else [y, norm(y, case["pre"], "pre")]
        if back:
            seeds = [cut("dy")] if case["pre"] == "none" else [cut("dy"), cut("dn")]
            all_ = torch.autograd.grad(got, leaves + list(par.values()), seeds)
            got = list(all_[:len(leaves)])
            sums = [a + g for a, g in zip(sums, all_[len(leaves):])]
        if rows_out is None:
            rows_out = [torch.empty(case["rows"], case["dim"], dtype=torch.float64, device=DEV) for _ in got]
        for o, g in zip(rows_out, got):
            o[r0:r0 + step] = g.detach()
    if back:
        return rows_out + sums
    return rows_out[0] if len(rows_out) == 1 else tuple(rows_out)
