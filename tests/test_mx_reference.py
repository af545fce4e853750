"""The references of the norm and MX tests, against hand-worked values and
against differences (CPU)."""
import numpy as np

import mx_reference as R


def test_formats_by_hand():
    assert R.E2M1.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6]
    assert R.E4M3[[1, 8, 126]].tolist() == [2.0 ** -9, 2.0 ** -6, 448] and len(R.E4M3) == 127
    x = np.zeros((1, 40))
    # 6.5 -> scale 2^0; ties 2.5 -> 2, 5 -> 4, 0.25 -> 0, 0.75 -> 1, 1.25 -> 1; 6.5 saturates
    x[0, :8] = [6.5, 2.5, -5, 0.25, 0.75, 1.25, -3.5, 0]
    x[0, 32:36] = [48, 16, -4, 1]       # floor(log2 48) - 2 = 3: 6, 2, -0.5, 0.125 -> 0
    c, s = R.mx_quantize(x, "mxfp4")
    assert s.tolist() == [[127, 130]]
    assert R.mx_values(c, s, "mxfp4")[0, [0, 1, 2, 3, 4, 5, 6, 7, 32, 33, 34, 35]].tolist() == \
        [6, 2, -4, 0, 1, 1, -4, 0, 48, 16, -4, 0]
    c, s = R.mx_quantize(np.array([[500.0, 17, 2.0 ** -10, np.nextafter(2.0 ** -10, 1)]]), "mxfp8")
    assert s[0, 0] == 127 and c[0, :4].tolist() == [126, 0x58, 0, 1]   # 500 saturates, 17 ties to 16


def test_zero_nan_and_tiny_blocks():
    x = np.zeros((3, 32))
    x[1, 3] = np.nan
    x[2, 0] = 2.0 ** -140
    c, s = R.mx_quantize(x, "mxfp4")
    assert s.tolist() == [[0], [255], [0]] and not c.any()
    assert np.isnan(R.mx_values(c, s, "mxfp4")[1]).all()


def test_pack_round_trip():
    c = np.arange(64, dtype=np.uint8).reshape(2, 32) % 16
    assert (R.unpack(R.pack(c)) == c).all() and R.pack(c)[0, 0] == 0x10


def test_gradient_against_differences():
    rng = np.random.default_rng(5)
    h, w, dy = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7))
    eps, d = 1e-3, 1e-6
    f = lambda h, w: (dy * h * R.rstd(h, eps)[:, None] * w).sum()   # noqa: E731
    dx, dw = R.grad(dy, h, w, R.rstd(h, eps))
    for i in range(3):
        for j in range(7):
            e = np.zeros((3, 7))
            e[i, j] = d
            assert abs((f(h + e, w) - f(h - e, w)) / (2 * d) - dx[i, j]) < 1e-7
    for j in range(7):
        e = np.zeros(7)
        e[j] = d
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * d) - dw[j]) < 1e-7
