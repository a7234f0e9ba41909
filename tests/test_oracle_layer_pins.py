"""Pins of the float64 oracle of the operators around the scan: closed forms
and special cases for the forwards, central differences for the backwards."""
import numpy as np
import pytest

from oracle import layer as O


def rand(seed, *shape):
    return np.random.default_rng(seed).normal(0, 1, shape)


def difference(f, a, d, h=1e-5):
    return (f(a + h * d) - f(a - h * d)) / (2 * h)


def assert_gradients(loss, args, grads, seed):
    """loss(**args) against grads along random directions.  Central differences of step h are off
    by h^2 / 6 of the third derivative and 2^-52 / h of the loss: 1e-6 of the scale covers both."""
    rng = np.random.default_rng(seed)
    for name, g in grads.items():
        d = rng.normal(0, 1, args[name].shape)
        num = difference(lambda v: loss(**{**args, name: v}), args[name], d)
        assert abs(num - (g * d).sum()) <= 1e-6 * (abs(num) + np.abs(g * d).sum()), name


def test_conv_is_numpys_convolution():
    x, w = rand(0, 2, 9, 3), rand(1, 3, 4)
    y, final = O.conv1d(x, w, act=False)
    for b in range(2):
        for c in range(3):
            np.testing.assert_allclose(y[b, :, c], np.convolve(x[b, :, c], w[c, ::-1])[:9], rtol=1e-13, atol=1e-13)
    assert np.array_equal(final, x[:, 6:])


@pytest.mark.parametrize("L", [0, 1, 2, 7])
def test_conv_in_two_calls_is_one(L):
    x, w, bias, init = rand(2, 2, L + 4, 3), rand(3, 3, 4), rand(4, 3), rand(5, 2, 3, 3)
    y, final = O.conv1d(x, w, bias, init)
    y1, f1 = O.conv1d(x[:, :L], w, bias, init)
    y2, f2 = O.conv1d(x[:, L:], w, bias, f1)
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(f2, final)


def test_conv_padding_is_a_shorter_sequence():
    x, w, bias, init = rand(6, 3, 6, 2), rand(7, 2, 3), rand(8, 2), rand(9, 3, 2, 2)
    y, final = O.conv1d(x, w, bias, init, pad=[0, 2, 6])
    y2, f2 = O.conv1d(x[1:2, 2:], w, bias, init[1:2])
    assert np.array_equal(y[1, 2:], y2[0]) and not y[1, :2].any() and np.array_equal(final[1], f2[0])
    assert not y[2].any() and np.array_equal(final[2], init[2])


def test_selective_scan_with_equal_decays_is_the_scalar_recurrence():
    """A equal over states and channels of a head is the chunked scan's recurrence."""
    import oracle
    b, L, H, P, N, G = 2, 7, 2, 4, 3, 1
    x, B, C = rand(10, b, L, H, P), rand(11, b, L, G, N), rand(12, b, L, G, N)
    dt, A, D, bias = rand(13, b, L, H), -np.abs(rand(14, H)), rand(15, H), rand(16, H)
    y, fs = oracle.recurrent(x, dt, bias, A, B, C, D)
    wide = lambda v: np.repeat(v, P, -1)
    y2, f2 = O.selective_scan(x.reshape(b, L, H * P), wide(dt), wide(bias), np.repeat(wide(A)[:, None], N, 1), B, C,
                              wide(D))
    np.testing.assert_allclose(y2.reshape(y.shape), y, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(f2.reshape(b, H, P, N).transpose(0, 1, 3, 2), fs, rtol=1e-12, atol=1e-12)


def test_selective_scan_in_two_calls_and_padded():
    b, L, D, G, N = 2, 6, 4, 2, 3
    a = dict(x=rand(20, b, L, D), dt_raw=rand(21, b, L, D), dt_bias=rand(22, D), A=-np.abs(rand(23, D, N)),
             B=rand(24, b, L, G, N), C=rand(25, b, L, G, N), D=rand(26, D), z=rand(27, b, L, D))
    init = rand(28, b, D, N)
    cut = lambda lo, hi: {k: v[:, lo:hi] if v.ndim > 2 and k != "A" else v for k, v in a.items()}
    y, f = O.selective_scan(**a, init=init)
    y1, f1 = O.selective_scan(**cut(0, 2), init=init)
    y2, f2 = O.selective_scan(**cut(2, L), init=f1)
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(f, f2)
    yp, fp = O.selective_scan(**a, init=init, pad=[2, 6])
    y3, f3 = O.selective_scan(**cut(2, L), init=init)
    assert np.array_equal(yp[0, 2:], y3[0]) and np.array_equal(fp[0], f3[0]) and not yp[0, :2].any()
    assert np.array_equal(fp[1], init[1]) and not yp[1].any()


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("L", [1, 5])
def test_conv_gradients_by_differences(act, L):
    args = dict(x=rand(30, 2, L, 3), weight=rand(31, 3, 4), bias=rand(32, 3), init=rand(33, 2, 3, 3))
    dy, df = rand(34, 2, L, 3), rand(35, 2, 3, 3)

    def loss(**a):
        y, f = O.conv1d(**a, act=act)
        return (y * dy).sum() + (f * df).sum()

    g = O.conv1d_bwd(**args, dy=dy, dfinal=df, act=act)
    assert_gradients(loss, args, {"x": g["dx"], "weight": g["dweight"], "bias": g["dbias"], "init": g["dinit_state"]}, 36)


@pytest.mark.parametrize("gate", [True, False])
def test_selective_scan_gradients_by_differences(gate):
    b, L, D, G, N = 2, 5, 4, 2, 3
    args = dict(x=rand(40, b, L, D), dt_raw=rand(41, b, L, D), dt_bias=rand(42, D), A=-np.abs(rand(43, D, N)),
                B=rand(44, b, L, G, N), C=rand(45, b, L, G, N), D=rand(46, D), z=rand(47, b, L, D) if gate else None,
                init=rand(48, b, D, N))
    dy, df = rand(49, b, L, D), rand(50, b, D, N)

    def loss(**a):
        y, f = O.selective_scan(**a)
        return (y * dy).sum() + (f * df).sum()

    g = O.selective_scan_bwd(**args, dy=dy, dfinal=df)
    grads = {"x": g["dx"], "dt_raw": g["ddt_raw"], "dt_bias": g["ddt_bias"], "A": g["dA"], "B": g["dB"], "C": g["dC"],
             "D": g["dD"], "init": g["dinit_state"]}
    assert_gradients(loss, args, {**grads, **({"z": g["dz"]} if gate else {})}, 51)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("act", ["none", "silu", "after", "before"])
def test_group_norm_gradients_by_differences(center, act):
    args = dict(x=rand(60, 4, 12), weight=rand(61, 12), bias=rand(62, 12),
                z=rand(63, 4, 12) if act in ("after", "before") else None)
    rest = dict(ngroups=3, eps=1e-3, center=center, act=act)
    dy = rand(64, 4, 12)
    g = O.group_norm_bwd(**args, dy=dy, **rest)
    grads = {"x": g["dx"], "weight": g["dweight"], "bias": g["dbias"]}
    assert_gradients(lambda **a: (O.group_norm(**a, **rest) * dy).sum(), args,
                     {**grads, **({"z": g["dz"]} if args["z"] is not None else {})}, 65)


def test_group_norm_closed_form():
    x = np.array([[3.0, 4.0, 1.0, 1.0]])
    y = O.group_norm(x, None, None, None, 2, 1e-300, False, "none")
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), 4 / np.sqrt(12.5), 1, 1]], rtol=1e-15)
    y = O.group_norm(x, None, None, None, 2, 0.25, True, "none")
    np.testing.assert_allclose(y, [[-0.5 / np.sqrt(0.5), 0.5 / np.sqrt(0.5), 0, 0]], rtol=1e-15)
