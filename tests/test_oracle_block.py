"""oracle.block against closed forms and central finite differences."""
import numpy as np
import pytest

from oracle import block


def _differences(fn, x, eps=1e-6):
    """Central differences of a scalar function of an array."""
    g = np.zeros_like(x)
    for k in np.ndindex(x.shape):
        keep = x[k]
        x[k] = keep + eps
        up = fn()
        x[k] = keep - eps
        g[k] = (up - fn()) / (2 * eps)
        x[k] = keep
    return g


def _scan_inputs(gate, igate, rng, B=2, T=5, C=3):
    f = rng.normal(size=(B, T, C))
    return dict(x=rng.normal(size=(B, T, C)), f=-np.abs(f) if gate == "log" else f,
                i=rng.normal(size=(B, T, C)) if igate else None, decay=rng.uniform(0.1, 2.0, C) if gate == "power" else None,
                h0=rng.normal(size=(B, C)))


@pytest.mark.parametrize("igate", [False, True])
@pytest.mark.parametrize("gate", ["log", "sigmoid", "power"])
def test_scan_gradients_are_those_of_differences(gate, igate):
    rng = np.random.default_rng(1)
    v = _scan_inputs(gate, igate, rng)
    d_h, d_end, lens = rng.normal(size=v["x"].shape), rng.normal(size=v["h0"].shape), [5, 3]
    kw = dict(gate=gate, decay=v["decay"], h0=v["h0"], lens=lens)

    def loss():
        h, end = block.scan_forward(v["x"], v["f"], v["i"], gate=gate, decay=v["decay"], h0=v["h0"], lens=lens)
        return (h * d_h).sum() + (end * d_end).sum()

    got = block.scan_backward(v["x"], v["f"], v["i"], d_h=d_h, dh_final=d_end, **kw)
    for n in ("x", "f", "i", "decay", "h0"):
        if v[n] is not None:
            np.testing.assert_allclose(got["d" + n], _differences(loss, v[n]), rtol=2e-7, atol=2e-8, err_msg=n)


def test_scan_closed_forms():
    T = 40
    x, f = np.ones((1, T, 8)), np.full((1, T, 8), np.log(0.9))
    h, end = block.scan_forward(x, f, gate="log")          # a geometric sum
    np.testing.assert_allclose(h[0, :, 0], (1 - 0.9 ** np.arange(1, T + 1)) / 0.1, rtol=1e-12)
    np.testing.assert_array_equal(end[0], h[0, -1])
    f = np.full((1, T, 8), 1.3)
    h, _ = block.scan_forward(x, f, gate="sigmoid", h0=np.ones((1, 8)))   # a mean of ones stays one
    np.testing.assert_allclose(h, 1.0, rtol=1e-13)
    # the power gate keeps the variance: a^2 + m^2 = 1
    a, m = block._gates(np.linspace(-9, 9, 50), "power", 0.7)
    np.testing.assert_allclose(a * a + m * m, 1.0, rtol=1e-14)
    # cut in two, the second part going on from the state of the first
    rng = np.random.default_rng(2)
    v = _scan_inputs("power", True, rng, T=9)
    whole, end = block.scan_forward(v["x"], v["f"], v["i"], gate="power", decay=v["decay"], h0=v["h0"])
    one, mid = block.scan_forward(v["x"][:, :4], v["f"][:, :4], v["i"][:, :4], gate="power", decay=v["decay"], h0=v["h0"])
    two, last = block.scan_forward(v["x"][:, 4:], v["f"][:, 4:], v["i"][:, 4:], gate="power", decay=v["decay"], h0=mid)
    np.testing.assert_array_equal(np.concatenate((one, two), 1), whole)
    np.testing.assert_array_equal(last, end)


@pytest.mark.parametrize("activation", ["silu", None])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_gradients_are_those_of_differences(W, activation):
    rng = np.random.default_rng(3)
    B, T, C = 3, 5, 2
    v = dict(x=rng.normal(size=(B, T, C)), w=rng.normal(size=(C, W)), bias=rng.normal(size=C), s0=rng.normal(size=(B, W - 1, C)))
    d_y, d_s, lens = rng.normal(size=(B, T, C)), rng.normal(size=(B, W - 1, C)), [5, 1, 0]

    def loss():
        y, end = block.conv_forward(v["x"], v["w"], v["bias"], activation=activation, s0=v["s0"], lens=lens)
        return (y * d_y).sum() + (end * d_s).sum()

    got = block.conv_backward(v["x"], v["w"], v["bias"], d_y=d_y, activation=activation, s0=v["s0"], ds_final=d_s, lens=lens)
    for n in v:
        np.testing.assert_allclose(got["d" + n], _differences(loss, v[n]), rtol=2e-7, atol=2e-8, err_msg=n)


def test_conv_is_numpys_convolution():
    rng = np.random.default_rng(4)
    x, w = rng.normal(size=(1, 11, 2)), rng.normal(size=(2, 4))
    y, end = block.conv_forward(x, w, activation=None)
    for c in range(2):
        np.testing.assert_allclose(y[0, :, c], np.convolve(x[0, :, c], w[c, ::-1])[:11], rtol=1e-12, atol=1e-14)
    np.testing.assert_array_equal(end, x[:, -3:])


@pytest.mark.parametrize("activation", ["silu", "sigmoid", None])
@pytest.mark.parametrize("post", [False, True])
def test_block_norm_gradients_are_those_of_differences(post, activation):
    rng = np.random.default_rng(5)
    shape, C = (2, 3, 4), 4
    v = dict(residual=rng.normal(size=shape), y=rng.normal(size=shape), gate=rng.normal(size=shape) if activation else None,
             weight=rng.normal(size=C), post_weight=rng.normal(size=C) if post else None, scale=rng.normal(size=C))
    up = dict(d_residual_out=rng.normal(size=shape), d_out=rng.normal(size=shape))
    kw = dict(post_norm=post, activation=activation or "sigmoid", residual_scale=0.7, eps=1e-2)

    def loss():
        r, n = block.block_norm(**v, **kw)
        return (r * up["d_residual_out"]).sum() + (n * up["d_out"]).sum()

    g = block.block_norm(**v, **kw, **up)[2]
    names = dict(residual="dr", y="dy", gate="dgate", weight="dw", post_weight="dw_post", scale="dscale")
    for n, d in names.items():
        if v[n] is not None:
            np.testing.assert_allclose(g[d], _differences(loss, v[n]), rtol=5e-7, atol=5e-8, err_msg=n)


def test_block_norm_of_unit_rows():
    r, n = block.block_norm(np.full((1, 1, 4), 3.0), eps=0.0)
    np.testing.assert_allclose(r, 3.0)
    np.testing.assert_allclose(n, 1.0)
    r, n = block.block_norm(np.zeros((1, 1, 4)), np.full((1, 1, 4), -2.0), post_norm=True, scale=np.full(4, 0.5), eps=0.0)
    np.testing.assert_allclose(r, -0.5)
