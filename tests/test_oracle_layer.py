"""The float64 definitions of the layer operators, pinned by closed forms and by central
differences (no GPU)."""
import numpy as np
import pytest

import oracle
from oracle import layer


def _inputs(seed, B=2, T=5, H=4, Hk=2, dk=3, dv=4):
    r = np.random.default_rng(seed)
    g = -r.uniform(0.01, 1.0, H)
    return (r.standard_normal((B, T, Hk, dk)), r.standard_normal((B, T, Hk, dk)), r.standard_normal((B, T, H, dv)), g,
            r.standard_normal((B, H, dk, dv)), r.standard_normal((B, T, H, dv)), r.standard_normal((B, H, dk, dv)))


def test_linear_forward_is_the_decayed_sum():
    q, k, v, g, s0, _, _ = _inputs(0)
    o, S = layer.linear_forward(q, k, v, g, s0)
    b, h, t = 1, 3, 4
    want = np.exp(g[h] * (t + 1)) * s0[b, h]
    for j in range(t + 1):
        want = want + np.exp(g[h] * (t - j)) * np.outer(k[b, j, 1], v[b, j, h])
    np.testing.assert_allclose(S[b, h], want, rtol=1e-13)
    np.testing.assert_allclose(o[b, t, h], want.T @ q[b, t, 1], rtol=1e-12)


def test_linear_forward_is_asym_without_its_erase():
    """S <- S D + k (eta v)^T with j = 0 and eta = 1 is the same recurrence."""
    q, k, v, g, s0, _, _ = _inputs(1, H=2, Hk=2)
    B, T, H, dk = k.shape
    inp = dict(variant="asym", B=B, T=T, H=H, dk=dk, dv=v.shape[3], n_h=1, dtype="f32", q=q, k=k, v=v,
               alpha=np.broadcast_to(np.exp(g)[:, None], k.shape), j=np.zeros_like(k), eta=np.ones((B, T, H)))
    o_ref, S_ref = oracle.forward(inp, s0)
    o, S = layer.linear_forward(q, k, v, g, s0)
    np.testing.assert_allclose(o, o_ref, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S, S_ref, rtol=1e-12, atol=1e-12)


def test_linear_lengths():
    q, k, v, g, s0, _, _ = _inputs(2)
    keep = np.full(v.shape, 7.0)
    o, S = layer.linear_forward(q, k, v, g, s0, lens=[0, 3], o=keep)
    assert np.all(o[0] == 7.0) and np.all(o[1, 3:] == 7.0) and np.array_equal(S[0], s0[0])
    o2, S2 = layer.linear_forward(q[1:, :3], k[1:, :3], v[1:, :3], g, s0[1:])
    np.testing.assert_array_equal(o[1, :3], o2[0])
    np.testing.assert_array_equal(S[1], S2[0])


def _differences(f, x, eps=1e-6):
    out = np.zeros_like(x)
    flat, grad = x.reshape(-1), out.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + eps
        up = f()
        flat[i] = keep - eps
        grad[i] = (up - f()) / (2 * eps)
        flat[i] = keep
    return out


@pytest.mark.parametrize("lens", [None, [2, 4]])
def test_linear_backward_against_differences(lens):
    q, k, v, g, s0, do, ds = _inputs(3, T=4)

    def loss():
        o, S = layer.linear_forward(q, k, v, g, s0, lens=lens)
        return float((o * do).sum() + (S * ds).sum())
    got = layer.linear_backward(q, k, v, g, do, s0, ds, lens=lens)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("ds0", s0)):
        np.testing.assert_allclose(got[name], _differences(loss, x), rtol=1e-6, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_norm_against_differences(norm, interleaved):
    r = np.random.default_rng(4)
    x, w, dy = r.standard_normal((2, 3, 2, 8)), r.standard_normal(8), r.standard_normal((2, 3, 2, 8))
    a = r.uniform(-3, 3, (9, 2))
    kw = dict(norm=norm, eps=0.3, scale=0.7, cos=np.cos(a), sin=np.sin(a), positions=r.integers(0, 9, (2, 3)),
              interleaved=interleaved)
    y, dx, dw = layer.head_norm(x, w, dy=dy, **kw)
    loss = lambda: float((layer.head_norm(x, w, **kw) * dy).sum())  # noqa: E731
    np.testing.assert_allclose(dx, _differences(loss, x), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dw, _differences(loss, w), rtol=1e-6, atol=1e-8)
    # a rotation keeps norms, and L2 rows without weights have norm |x| / sqrt(|x|^2 + eps)
    plain = layer.head_norm(x, None, **{**kw, "scale": 1.0})
    sq = (x * x).sum(-1)
    want = sq / ((sq / 8 if norm == "rms" else sq) + 0.3)
    np.testing.assert_allclose((plain * plain).sum(-1), want, rtol=1e-12)


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
def test_gated_norm_against_differences(activation):
    r = np.random.default_rng(5)
    x, z, w, dy = (r.standard_normal(s) for s in ((1, 3, 2, 8), (1, 3, 2, 8), (8,), (1, 3, 2, 8)))
    kw = dict(eps=0.2, activation=activation)
    _, dx, dz, dw = layer.gated_norm(x, z, w, dy=dy, **kw)
    loss = lambda: float((layer.gated_norm(x, z, w, **kw) * dy).sum())  # noqa: E731
    for got, leaf in ((dx, x), (dz, z), (dw, w)):
        np.testing.assert_allclose(got, _differences(loss, leaf), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("n", [0, 1, 2, 9])
@pytest.mark.parametrize("log_decay", [-0.3, float("-inf")])
def test_the_gradients_recurrence_as_the_header_states_it(log_decay, n):
    """G_n = d_s_final + q_n do_n^T, undecayed, then G_t = e^g G_{t+1} + q_t do_t^T; ds0 = e^g G_1,
    or d_s_final itself for a sequence of no tokens."""
    rng = np.random.default_rng(n)
    q, k, v, do = (rng.standard_normal((1, 9, 1, d)) for d in (4, 4, 3, 3))
    ds = rng.standard_normal((1, 1, 4, 3))
    got = layer.linear_backward(q, k, v, [log_decay], do, ds_final=ds, lens=[n])
    G, gam = ds[0, 0], np.exp(log_decay)
    for t in range(n - 1, -1, -1):
        G = (G if t == n - 1 else gam * G) + np.outer(q[0, t, 0], do[0, t, 0])
        np.testing.assert_allclose(got["dk"][0, t, 0], G @ v[0, t, 0], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(got["dv"][0, t, 0], G.T @ k[0, t, 0], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(got["ds0"][0, 0], gam * G if n else ds[0, 0], rtol=1e-12, atol=1e-12)
