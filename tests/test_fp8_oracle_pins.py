"""Pins of the 8-bit path's oracle (CPU): the number format against torch's,
the scale rule by its definition, the products by sums in plain Python, the
norm's gradient by differences."""

import math

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O


def test_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, O.E4M3, equal_nan=True)
    assert np.nanmax(O.E4M3) == 448


def test_encoding_is_torchs():
    rng = np.random.default_rng(1)
    v = (rng.standard_normal(20000) * np.exp2(rng.integers(-12, 7, 20000))).astype(np.float32)
    ties = (O.E4M3[:126] + O.E4M3[1:127]) / 2  # every midpoint
    v = np.concatenate([v[np.abs(v) <= 448], ties, -ties, O.E4M3[:127], [0.0, -0.0]]).astype(np.float32)
    got = O.e4m3_encode(v)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, want)
    assert O.e4m3_encode([np.nan, np.inf, -np.inf]).tolist() == [0x7F] * 3


@pytest.mark.parametrize("a", [0.0, 1e-45, 2.0**-127, 448 * 2.0**-126, 448 * 2.0**-126 * 1.0000001, 1.0, 447.9, 448.0, 448.1, 896.0, 3.4e38])
def test_scale_is_the_smallest_power(a):
    p = float(O.power(O.scale_byte(a)))
    assert a <= 448 * p
    assert p == 2.0**-126 or a > 448 * p / 2
    assert math.frexp(p)[0] == 0.5


def test_rows_and_weight_by_hand():
    x = np.zeros((2, 130))
    x[0, 0], x[0, 128], x[1, 1] = 448.0, -3.5, np.inf
    q, s = O.quant_rows(x)
    assert q.shape == (2, 256) and s.shape == (2, 4)
    # 448 = 448 * 1; 3.5 = 448 / 128, so its group's scale is 2^-7; padding: ones
    assert s[0].tolist() == [127, 120, 127, 127] and s[1].tolist() == [1, 1, 127, 127]
    assert O.E4M3[q[0, 0]] == 448 and O.E4M3[q[0, 128]] == -448 and np.isnan(O.E4M3[q[1, 1]])
    assert np.array_equal(np.nan_to_num(O.wide_rows(q, s))[0, [0, 128]], [448.0, -3.5])
    w = np.zeros((129, 5))
    w[0, 0], w[128, 4] = 1.0, 896.0
    q, s = O.quant_weight(w)
    assert q.shape == (129, 128) and s.shape == (2, 4)
    assert np.array_equal(O.wide_weight(q, s)[[0, 128], [0, 4]], [1.0, 896.0])


def test_products_by_sums():
    rng = np.random.default_rng(2)
    x, w, b = rng.standard_normal((3, 256)), rng.standard_normal((2, 4, 256)), rng.standard_normal((2, 4))
    y, scale = O.linear(x, w[0], b[0])
    for m in range(3):
        for n in range(4):
            assert abs(y[m, n] - math.fsum([*(x[m] * w[0, n]), b[0, n]])) < 1e-12
            assert abs(scale[m, n] - math.fsum(abs(x[m] * w[0, n]))) < 1e-12
    rows = np.array([2, 0, 2, 1, 0])
    ye, _ = O.experts(x, rows, [0, 3, 4], w, b)
    assert ye.shape == (4, 4)
    for r in range(4):
        e = 0 if r < 3 else 1
        assert np.allclose(ye[r], O.linear(x[rows[r]][None], w[e], b[e])[0][0], atol=1e-12)


def test_norm_gradient_by_differences():
    rng = np.random.default_rng(3)
    h, w, dy, dh = rng.standard_normal((2, 7)), rng.standard_normal(7), rng.standard_normal((2, 7)), rng.standard_normal((2, 7))
    _, r = O.rms_norm(h, w, 1e-3)
    dx, dw = O.rms_norm_bwd(dy, h, w, r, dh)

    def loss(h, w):
        return (O.rms_norm(h, w, 1e-3)[0] * dy).sum() + (h * dh).sum()

    d = 1e-6
    for i in range(2):
        for k in range(7):
            e = np.zeros_like(h)
            e[i, k] = d
            assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - dx[i, k]) < 1e-8
    for k in range(7):
        e = np.zeros(7)
        e[k] = d
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - dw[k]) < 1e-8
