"""Pins for the 4-bit oracle (CPU): rounding against a search over all levels and against ties by
hand, the scales against their definitions, and the gated block's gradients against differences."""
import numpy as np
import pytest

from oracle import mx4


def test_e2m1_ties_and_saturation():
    # halfway points go to the level whose mantissa bit is 0
    ties = {0.25: 0.0, 0.75: 1.0, 1.25: 1.0, 1.75: 2.0, 2.5: 2.0, 3.5: 4.0, 5.0: 4.0}
    for v, want in ties.items():
        assert mx4.LEVELS[mx4.e2m1_round(v)] == want
        assert mx4.LEVELS[mx4.e2m1_round(np.nextafter(v, 9))] > v
        assert mx4.LEVELS[mx4.e2m1_round(np.nextafter(v, 0))] < v
    assert mx4.LEVELS[mx4.e2m1_round(6.0)] == 6 and mx4.LEVELS[mx4.e2m1_round(1e30)] == 6


def test_mxfp4_scale_is_a_power_of_two_that_saturates_at_most_a_quarter():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(64, 160)) * np.exp2(rng.integers(-20, 20, size=(64, 1)))
    codes, byte, val = mx4.quantize(x, "mxfp4")
    pad = np.zeros((64, 256))
    pad[:, :160] = x
    top = np.abs(pad.reshape(64, -1, 32)).max(-1)
    s = np.exp2(byte.astype(float) - 127)
    live = top > 0
    assert ((top / s)[live] >= 4).all() and ((top / s)[live] < 8).all()
    assert (byte[~live] == 0).all()
    # below 6 s an element is within half a level's step (at most s) of x, above it becomes 6 s
    err = np.abs(val - x)
    lim = np.repeat(s, 32, 1)[:, :160]
    assert (err <= np.where(np.abs(x) <= 6 * lim, lim, np.abs(x) - 6 * lim) * (1 + 1e-12)).all()


@pytest.mark.parametrize("f", [1.0, 2.0 ** -9])
def test_nvfp4_scale_bytes_decode_to_the_rounded_scale(f):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(32, 128)) * np.exp2(rng.integers(-8, 6, size=(32, 1))) * f
    _, byte, val = mx4.quantize(x, "nvfp4", f)
    e, m = byte.astype(int) >> 3, byte.astype(int) & 7
    s = np.where(e > 0, (8 + m) * np.exp2(e - 10.0), m * 2.0 ** -9)
    want = np.abs(x.reshape(32, 8, 16)).max(-1) / (6 * f)
    assert (np.abs(s - want) <= np.maximum(want * 2.0 ** -4, 2.0 ** -10)).all()
    assert (np.abs(val) <= np.repeat(s, 16, 1) * 6 * f).all()


def test_factor_reaches_the_largest_product_and_no_further():
    for amax in (2688.0, 2688.0 * 2 ** -7, 2689.0, 1.0, 3e-30, 1e30):
        got, f = mx4.tensor_factor(np.array([[amax, -amax / 2]]))
        assert got == amax and f / 2 * 2688 < amax <= f * 2688
    assert mx4.tensor_factor(np.zeros((2, 3))) == (0.0, 1.0)


def test_non_finite_blocks():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.inf, np.nan
    codes, byte, val = mx4.quantize(x, "mxfp4")
    assert byte[0, 0] == 255 and byte[1, 1] == 255 and byte[0, 1] == 125
    assert np.isnan(val[0, :32]).all() and np.isfinite(val[0, 32:]).all()
    assert not codes[0, :32].any()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradients_match_differences(name):
    rng = np.random.default_rng(3)
    da, g, u = (rng.normal(size=(5, 7)) for _ in range(3))
    dg, du, a = mx4.gated_bwd(da, g, u, name)
    loss = lambda g, u: float((da * mx4.act(g, name)[0] * u).sum())  # noqa: E731
    assert np.allclose(a, mx4.act(g, name)[0] * u)
    h = 1e-5  # central differences: error h^2 |f'''| / 6 + rounding eps / h, both below 1e-9
    for i in range(5):
        for j in range(7):
            e = np.zeros((5, 7))
            e[i, j] = h
            assert abs((loss(g + e, u) - loss(g - e, u)) / (2 * h) - dg[i, j]) < 1e-8
            assert abs((loss(g, u + e) - loss(g, u - e)) / (2 * h) - du[i, j]) < 1e-8


def test_tanh_gelu_keeps_its_negative_tail():
    """(1 + tanh y) / 2 from decimal arithmetic at 60 digits, where 1 + tanh y cancels in 64 bits."""
    import decimal
    with decimal.localcontext(decimal.Context(prec=60)):
        for z in (-3.0, -6.0, -10.0):
            d = decimal.Decimal(z)
            pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")
            y = (2 / pi).sqrt() * (d + decimal.Decimal("0.044715") * d ** 3)
            want = d / (1 + (-2 * y).exp())
            assert abs(decimal.Decimal(float(mx4.act(z, "gelu_tanh")[0])) / want - 1) < 1e-13
