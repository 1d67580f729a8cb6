"""Pins of the oracle of the norm, the block quantisation and the products grouped by
expert: rounding against torch's CPU conversion, gradients against differences of the
forward form and against autograd, scales against their definition."""

import numpy as np
import pytest
import torch

from oracle import layer as ol


def test_e4m3_rounding_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    codes = np.unique(codes[np.isfinite(codes)]).astype(np.float64)
    mids = (codes[1:] + codes[:-1]) / 2
    v = np.concatenate([codes, mids, mids * (1 + 1e-6), mids * (1 - 1e-6),
                        np.random.default_rng(0).normal(size=4000) * 60, [448.0, -448.0, 2.0 ** -11]])
    v = np.clip(v.astype(np.float32), -448, 448)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ol.e4m3_round(v), want)
    assert np.isnan(ol.e4m3_round([np.nan]))[0]


@pytest.mark.parametrize("block_rows", [1, 128])
def test_scales_are_the_smallest_that_fit(block_rows):
    x = np.random.default_rng(1).normal(size=(130, 300)) * np.exp(np.random.default_rng(2).normal(size=(130, 1)) * 9)
    x[3, :] = 0
    x[4, 0], x[5, 0], x[6, 0] = 448.0, 448.1, 2.0 ** -130
    s = ol.block_scales(x, block_rows)
    assert s.shape == (-(-130 // block_rows), 3)
    wide = ol.expand(s, x.shape, block_rows)
    assert np.all(np.abs(x) <= 448 * wide) and np.all(np.log2(s) == np.rint(np.log2(s)))
    for i in range(s.shape[0]):
        for j in range(3):
            b = np.abs(x[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128])
            assert s[i, j] == 2.0 ** -126 or b.max() > 448 * s[i, j] / 2
    x[0, 0], x[1, 0] = np.inf, np.nan
    q, s = ol.quantize(x, 1)
    assert np.isnan(s[0, 0]) and np.isnan(s[1, 0]) and np.isfinite(s[2, 0]) and np.isnan(q[0, :128]).all()


@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradients_against_differences(residual):
    rng = np.random.default_rng(3)
    x, w, d = rng.normal(size=(4, 7)) * 2, rng.normal(size=7), rng.normal(size=(4, 7))
    dres = rng.normal(size=(4, 7)) if residual else None
    eps, h = 1e-3, 1e-6

    def loss(x, w):
        return (ol.rmsnorm(x, w, eps) * d).sum() + (0 if dres is None else (x * dres).sum())

    dx, dw = ol.rmsnorm_backward(x, w, d, eps, dres)
    for i in range(4):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = h
            assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(7):
        e = np.zeros_like(w)
        e[j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_norm_gradients_against_autograd():
    rng = np.random.default_rng(4)
    x, w, d = (torch.tensor(rng.normal(size=s), requires_grad=True) for s in ((5, 11), (11,), (5, 11)))
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5) * w
    (y * d.detach()).sum().backward()
    dx, dw = ol.rmsnorm_backward(x.detach().numpy(), w.detach().numpy(), d.detach().numpy(), 1e-5)
    np.testing.assert_allclose(dx, x.grad.numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-12, atol=1e-13)


def test_ragged_gradients_against_differences_and_untouched_rows():
    rng = np.random.default_rng(5)
    off = [1, 3, 3, 6]
    a, b, d = rng.normal(size=(8, 4)), rng.normal(size=(3, 5, 4)), rng.normal(size=(8, 5))
    before = rng.normal(size=(8, 5))

    def loss(a, b):
        return (ol.ragged(a, b, off, np.zeros((8, 5)))[1:6] * d[1:6]).sum()

    c = ol.ragged(a, b, off, before)
    np.testing.assert_array_equal(c[[0, 6, 7]], before[[0, 6, 7]])
    da, db = ol.ragged_dgrad(d, b, off, np.zeros((8, 4))), ol.ragged_wgrad(d, a, off)
    assert np.all(db[1] == 0) and np.all(da[[0, 6, 7]] == 0)
    h = 1e-6
    for idx in np.ndindex(a.shape):
        e = np.zeros_like(a)
        e[idx] = h
        assert abs((loss(a + e, b) - loss(a - e, b)) / (2 * h) - da[idx]) < 1e-7
    for idx in np.ndindex(b.shape):
        e = np.zeros_like(b)
        e[idx] = h
        assert abs((loss(a, b + e) - loss(a, b - e)) / (2 * h) - db[idx]) < 1e-7


def test_block_scaled_product_is_the_product_of_the_values():
    rng = np.random.default_rng(6)
    x, y = rng.normal(size=(3, 200)), rng.normal(size=(140, 200))
    (qx, sx), (qy, sy) = ol.quantize(x, 1), ol.quantize(y, 128)
    c, mag = ol.block_scaled_product(qx, sx, qy, sy)
    vx, vy = qx * ol.expand(sx, x.shape, 1), qy * ol.expand(sy, y.shape, 128)
    np.testing.assert_allclose(c, np.einsum("mk,nk->mn", vx, vy), rtol=1e-12, atol=1e-12)
    # each value is within half an e4m3 step of what it stands for
    assert np.all(np.abs(vx - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * ol.expand(sx, x.shape, 1)))
    assert np.all(mag >= np.abs(c))
