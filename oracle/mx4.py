"""Plain 64-bit forms of the operators around the attention (numpy): MXFP4
quantisation, operands and products, and the norms before and after a block.

Each is written from its definition: the quantiser picks the nearest point of
the scaled E2M1 grid (ties to the even index) by comparing distances, the
products are sums of decoded values, the norms and their gradients the
formulas.  The norms also return, for every result, a magnitude: the result
with every term taken by its absolute value and every statistic's sensitivity
to its inputs' magnitudes added.  An evaluation in a format with rounding unit
u whose longest chain of operations has length L is then within L u magnitude
of the result, to first order in u.
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_SCALE = 255


def ceil_div(a, b):
    return -(-a // b)


def quantize(x):
    """x [R, K] -> (codes uint8 [R, Kp] one per element, scale bytes [R, Kp / 32])."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    nb = ceil_div(k, 32)
    full = np.zeros((rows, nb * 32))
    full[:, :k] = x
    blocks = full.reshape(rows, nb, 32)
    bad = ~np.isfinite(blocks).all(-1)
    amax = np.abs(np.where(bad[..., None], 0.0, blocks)).max(-1)
    _, e = np.frexp(amax)                      # amax = m 2^e, m in [0.5, 1)
    X = np.where(amax > 0, np.clip(e - 3, -127, 127), -127)
    t = np.where(bad[..., None], 0.0, blocks) * np.exp2(-X.astype(np.float64))[..., None]
    mag = np.minimum(np.abs(t), 6.0)
    dist = np.abs(mag[..., None] - E2M1)
    near = dist == dist.min(-1, keepdims=True)
    # of two nearest points the one with the even index
    idx = np.where(near.sum(-1) == 2, 2 * ceil_div(near.argmax(-1), 2), near.argmax(-1))
    codes = (idx | (np.signbit(t).astype(np.int64) << 3)).astype(np.uint8)
    codes[bad] = 0
    scales = np.where(bad, NAN_SCALE, X + 127).astype(np.uint8)
    return codes.reshape(rows, nb * 32), scales


def values(codes, scales, k=None):
    """Decoded values of one-per-element codes [R, Kp] and scale bytes."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    unit = np.where(scales == NAN_SCALE, np.nan, np.exp2(scales.astype(np.float64) - 127))
    v = v * np.repeat(unit, 32, axis=1)
    return v if k is None else v[:, :k]


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out


def scale_index(rows, blocks):
    """Position of each (row, block) scale byte in the tiled buffer."""
    r, c = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    return ((r // 128) * ceil_div(blocks, 4) + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4


def scale_bytes(rows, blocks):
    return ceil_div(rows, 128) * ceil_div(blocks, 4) * 512


def tile_scales(scales):
    out = np.zeros(scale_bytes(*scales.shape), np.uint8)
    out[scale_index(*scales.shape)] = scales
    return out


def untile_scales(tiled, rows, blocks):
    return tiled[scale_index(rows, blocks)]


# ---------------------------------------------------------------------------
# norms before and after a block
# ---------------------------------------------------------------------------


def _norm(v, V, kind, eps):
    """v with magnitude V -> (hat, its magnitude, r, the relative magnitude of r)."""
    if kind == "layer":
        c = v - v.mean(1, keepdims=True)
        C = V + V.mean(1, keepdims=True)
    else:
        c, C = v, V
    r = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    rel = 1.0 + r * r * (np.abs(c) * C).mean(1, keepdims=True)
    hat = c * r
    return hat, r * C + np.abs(hat) * rel, r, rel


def _sigmoid(u):
    return 1.0 / (1.0 + np.exp(-u))


def _gate(kind, u):
    """act(u), act'(u) and their magnitudes."""
    if kind == "none":
        one = np.ones((1, 1))
        return one, 0 * one, one, 0 * one
    if kind == "identity":
        return u, np.ones_like(u), np.abs(u), np.ones_like(u)
    s = _sigmoid(u)
    if kind == "sigmoid":
        return s, s * (1 - s), s * (1 + np.abs(u)), (s + s * s) * (1 + np.abs(u))
    return (u * s, s * (1 + u * (1 - s)), np.abs(u) * s * (1 + np.abs(u)),
            s * (1 + 2 * np.abs(u)) * (1 + np.abs(u)))


def block_norm(x, block, gate=None, scale=None, post_gamma=None, post_beta=None, pre_gamma=None,
               pre_beta=None, post="rms", pre="rms", gate_kind="silu", eps=1e-5, dy=None, dn=None):
    """Results and magnitudes: {name: (value, magnitude)} with y, n and, given
    dy, the gradients x, block, gate, scale, post_gamma, ..., pre_beta."""
    f = lambda a: None if a is None else np.asarray(a, np.float64)
    x, b, u = f(x), f(block), f(gate)
    D = x.shape[1]
    vec = lambda a, absent: np.full((1, D), absent) if a is None else f(a)[None, :]
    s, pg, pb = vec(scale, 1.0), vec(post_gamma, 1.0), vec(post_beta, 0.0)
    qg, qb = vec(pre_gamma, 1.0), vec(pre_beta, 0.0)
    if post == "none":
        bh, BH, rb, relb = b, np.abs(b), 1.0, 1.0
    else:
        bh, BH, rb, relb = _norm(b, np.abs(b), post, eps)
    p, Pm = bh * pg + pb, BH * np.abs(pg) + np.abs(pb)
    a, da, A, dA = _gate(gate_kind, u)
    y, Y = x + s * a * p, np.abs(x) + np.abs(s) * A * Pm
    out = {"y": (y, Y)}
    if pre != "none":
        yh, YH, ry, rely = _norm(y, Y, pre, eps)
        out["n"] = (yh * qg + qb, YH * np.abs(qg) + np.abs(qb))
    if dy is None:
        return out

    def through(hat, HAT, r, rel, g, G, kind):
        t = g - hat * (g * hat).mean(1, keepdims=True)
        T = G + HAT * (G * HAT).mean(1, keepdims=True)
        if kind == "layer":
            t = t - g.mean(1, keepdims=True)
            T = T + G.mean(1, keepdims=True)
        return r * t, r * rel * T

    total = lambda v, V: (v.sum(0), V.sum(0))
    d, Dm = f(dy), np.abs(f(dy))
    if pre != "none":
        dn = f(dn)
        out["pre_gamma"] = total(dn * yh, np.abs(dn) * YH)
        out["pre_beta"] = total(dn, np.abs(dn))
        t, T = through(yh, YH, ry, rely, dn * qg, np.abs(dn * qg), pre)
        d, Dm = d + t, Dm + T
    out["x"] = (d, Dm)
    out["scale"] = total(d * a * p, Dm * A * Pm)
    dp, DP = d * s * a, Dm * np.abs(s) * A
    if post == "none":
        out["block"] = (dp, DP)
    else:
        out["post_gamma"] = total(dp * bh, DP * BH)
        out["post_beta"] = total(dp, DP)
        out["block"] = through(bh, BH, rb, relb, dp * pg, DP * np.abs(pg), post)
    if gate_kind != "none":
        out["gate"] = (d * s * p * da, Dm * np.abs(s) * Pm * dA)
    return out
