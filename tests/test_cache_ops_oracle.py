"""The plain forms of the preparation and cache operators, checked against
independent statements of the same things (no GPU needed)."""

import numpy as np
import pytest
import torch

import oracle.cache_ops as co


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(8, 8), (12, 6), (5, 2)])
def test_gradients_against_differences(D, rot, interleaved):
    rng = np.random.default_rng(D)
    x, dy = rng.standard_normal((2, 2, 3, D)), rng.standard_normal((2, 2, 3, D))
    w, f = 1 + 0.3 * rng.standard_normal(D), rng.uniform(0.01, 1, rot // 2)
    kw = dict(pos=np.array([[3, 4, 9], [0, 1, 70]]), inv_freq=f, interleaved=interleaved, norm=True, eps=0.1)
    dx, dw = co.norm_rope_backward(x, dy, weight=w, **kw)
    h = 1e-6
    for idx in [(0, 0, 0, 0), (1, 1, 2, D - 1), (0, 1, 1, rot - 1)]:
        d = np.zeros_like(x)
        d[idx] = h
        diff = ((co.norm_rope(x + d, weight=w, **kw) - co.norm_rope(x - d, weight=w, **kw)) * dy).sum() / (2 * h)
        assert abs(diff - dx[idx]) < 1e-8
    for e in range(D):
        d = np.zeros(D)
        d[e] = h
        diff = ((co.norm_rope(x, weight=w + d, **kw) - co.norm_rope(x, weight=w - d, **kw)) * dy).sum() / (2 * h)
        assert abs(diff - dw[e]) < 1e-8


def test_rotation_is_a_rotation():
    x = np.random.default_rng(0).standard_normal((1, 3, 8))
    f = np.array([1.0, 0.5, 0.1])
    y = co.rotate(x, [5, 6, 7], f, False)
    assert np.allclose(np.abs(y[..., :3] + 1j * y[..., 3:6]), np.abs(x[..., :3] + 1j * x[..., 3:6]))
    assert np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose(co.rotate(y, [5, 6, 7], f, False, -1.0), x)


def test_e4m3_rounding_is_the_types():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    vals = np.unique(codes[np.isfinite(codes)])
    mids = (vals[1:] + vals[:-1]) / 2
    probe = np.concatenate([vals, mids, np.random.default_rng(1).uniform(-448, 448, 20000),
                            np.random.default_rng(2).uniform(-0.05, 0.05, 20000)])
    want = torch.from_numpy(probe).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(co.e4m3_round(probe.astype(np.float32)), want)


def test_block_scale_brings_the_block_into_range():
    for amax in [448.0, 448.0000001, 1.0, 0.875 * 2.0 ** 5, 1.75, 1e-30, 3e38, 223.9]:
        s = co.block_scale(amax)
        assert np.log2(s) == np.rint(np.log2(s)) and 224.0 < amax / s <= 448.0
    assert co.block_scale(0.0) == 0.0 and co.block_scale(1e-45) == 2.0 ** -126


def test_append_keeps_what_it_does_not_name():
    rng = np.random.default_rng(3)
    pool, scale = co.e4m3_round(rng.uniform(-400, 400, (4, 2, 8, 4))), np.full((4, 2, 2), 0.5)
    before, s_before = pool.copy(), scale.copy()
    rows = rng.standard_normal((2, 3, 4)) * 1000  # larger than 448 * 0.5: the block's scale grows
    co.append(rows, pool, scale, 4, [2, 0], 8, 6, 3)  # slots 6, 7 of page 2 and slot 0 of page 0
    assert np.array_equal(pool[[1, 3]], before[[1, 3]]) and np.array_equal(pool[2, :, :4], before[2, :, :4])
    assert np.array_equal(pool[0, :, 1:], before[0, :, 1:])
    assert np.array_equal(scale[2, :, 0], s_before[2, :, 0]) and np.all(scale[2, :, 1] > 0.5)
    # older tokens of the grown block stand for the same values within a step
    v0, v1 = before[2, :, 4:6] * 0.5, pool[2, :, 4:6] * scale[2, :, 1][:, None, None]
    assert np.all(np.abs(v0 - v1) <= 0.5 * co.e4m3_step(v0 / scale[2, :, 1][:, None, None]) * scale[2, :, 1][:, None, None])
