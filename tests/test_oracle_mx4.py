"""The 64-bit forms of the operators around the attention, pinned: the E2M1
grid point by point, the scale rule, the tiled scale layout, and the norms'
gradients against differences."""
import itertools

import numpy as np
import pytest

from oracle import mx4


def test_grid_and_ties():
    # one block per value, with 4.0 fixing the exponent 0: every midpoint goes
    # to the even neighbour, saturation above 5
    pts = mx4.E2M1
    mids = (pts[1:] + pts[:-1]) / 2
    for i, m in enumerate(mids):
        even = i if i % 2 == 0 else i + 1
        for t, want in ((m, even), (np.nextafter(m, 0), i), (np.nextafter(m, 9), i + 1)):
            x = np.zeros((1, 32))
            x[0, 0], x[0, 1], x[0, 2] = 4.0, t, -t
            codes, scales = mx4.quantize(x)
            assert scales[0, 0] == 127 and codes[0, 0] == 6
            assert codes[0, 1] == want and codes[0, 2] == want + 8
    x = np.zeros((1, 32))
    x[0, 0] = 7.99
    codes, scales = mx4.quantize(x)
    assert codes[0, 0] == 7 and scales[0, 0] == 127


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (1.0, 125), (1.99, 125), (2.0, 126), (4.0, 127),
                                       (2.0 ** -126, 0), (2.0 ** -125, 0), (2.0 ** -124, 1),
                                       (2.0 ** -140, 0), (2.0 ** 127, 252), (np.inf, 255), (np.nan, 255)])
def test_scale_bytes(amax, byte):
    x = np.zeros((1, 40))
    x[0, 5] = -amax
    codes, scales = mx4.quantize(x)
    assert scales[0, 0] == byte and scales[0, 1] == 0
    v = mx4.values(codes, scales, 40)
    assert np.isnan(v[0, :32]).all() if byte == 255 else np.abs(v - x).max() <= max(amax, 2.0 ** -126) / 4
    assert (v[0, 32:] == 0).all()


@pytest.mark.parametrize("rows,blocks", [(1, 1), (129, 5), (300, 9), (128, 4)])
def test_scale_layout_is_a_bijection_into_tiles(rows, blocks):
    at = mx4.scale_index(rows, blocks)
    assert len(np.unique(at)) == rows * blocks and at.max() < mx4.scale_bytes(rows, blocks)
    s = np.random.default_rng(0).integers(0, 255, (rows, blocks)).astype(np.uint8)
    assert np.array_equal(mx4.untile_scales(mx4.tile_scales(s), rows, blocks), s)
    # the four scales of 128 columns are one word; a tile's lanes are 16 bytes
    assert at[0, 0] == 0 and (blocks < 4 or at[0, 3] == 3)
    if rows > 33:
        assert at[1, 0] == 16 and at[32, 0] == 4


def _inputs(rng, R, D, post, pre, gate):
    v = lambda c=1.0: rng.normal(size=D) * 0.3 + c
    kw = dict(x=rng.normal(size=(R, D)), block=rng.normal(size=(R, D)) + 0.5,
              gate=rng.normal(size=(R, D)) if gate != "none" else None, scale=v(0.5),
              post_gamma=v() if post != "none" else None, post_beta=v(0) if post == "layer" else None,
              pre_gamma=v() if pre != "none" else None, pre_beta=v(0) if pre == "layer" else None)
    return kw


@pytest.mark.parametrize("post,pre,gate", list(itertools.product(("none", "rms", "layer"), ("none", "rms", "layer"),
                                                            ("none", "identity", "silu", "sigmoid"))))
def test_norm_gradients_match_differences(post, pre, gate):
    rng = np.random.default_rng(3)
    R, D = 3, 7
    kw = _inputs(rng, R, D, post, pre, gate)
    kinds = dict(post=post, pre=pre, gate_kind=gate, eps=1e-3)
    dy, dn = rng.normal(size=(R, D)), rng.normal(size=(R, D))

    def loss(**k):
        o = mx4.block_norm(**k, **kinds)
        return (o["y"][0] * dy).sum() + ((o["n"][0] * dn).sum() if pre != "none" else 0.0)

    got = mx4.block_norm(**kw, **kinds, dy=dy, dn=dn)
    h = 1e-5
    for name, t in kw.items():
        if t is None:
            continue
        g = got[name][0]
        assert g.shape == t.shape
        for at in np.ndindex(*t.shape):
            up, down = t.copy(), t.copy()
            up[at] += h
            down[at] -= h
            diff = (loss(**{**kw, name: up}) - loss(**{**kw, name: down})) / (2 * h)
            # central differences: h^2 times a third derivative, and 2^-53 / h of the loss
            assert abs(diff - g[at]) <= 1e-6 * (1 + abs(g[at])), (name, at)
    for v, mag in got.values():
        assert (np.abs(v) <= mag * (1 + 1e-12)).all()
