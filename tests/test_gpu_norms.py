"""Norms of queries and keys with the position rotation, and the gated norm, against their
float64 definitions (oracle.layer)."""
import numpy as np
import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu

# B, T, Hq, Hk, d, rot
QK = [
    (1, 1, 1, 1, 16, 16),
    (2, 37, 3, 1, 16, 8),
    (1, 65, 4, 2, 32, 0),
    (3, 19, 5, 5, 64, 64),
    (2, 70, 16, 8, 128, 64),
    (1, 300, 6, 3, 128, 128),
]


def _qk_case(case, dt, seed, fuse):
    from layer_util import DTYPES, dev, fused, rand
    B, T, Hq, Hk, d, rot = case
    gen = torch.Generator().manual_seed(seed)
    dtype = DTYPES[dt]
    q, k, pad = (rand(gen, (B, T, h, d), dtype, s) for h, s in ((Hq, 1.5), (Hk, 0.4), (1, 1.0)))
    wq, wk = (1 + rand(gen, (d,), torch.float32, 0.2) for _ in range(2))
    P = 2 * T + 3
    angle = torch.rand((P, max(rot // 2, 1)), generator=gen, dtype=torch.float64) * 6.3
    cos, sin = (angle.cos().float(), angle.sin().float()) if rot else (None, None)
    pos = torch.randint(0, P, (B, T), generator=gen, dtype=torch.int32) if rot else None
    dq, dk = rand(gen, (B, T, Hq, d), dtype), rand(gen, (B, T, Hk, d), dtype)
    host = dict(q=q, k=k, wq=wq, wk=wk, cos=cos, sin=sin, pos=pos, dq=dq, dk=dk)
    on = {n: None if t is None else t.to(dev()) for n, t in host.items()}
    if fuse:
        on["q"], on["k"], _ = fused([q, k, pad])
    return host, on


def _kw(t, norm, interleaved):
    return dict(norm=norm, eps=1e-5, q_scale=0.37, cos=t["cos"], sin=t["sin"], positions=t["pos"], interleaved=interleaved)


def _want(host, which, norm, interleaved, dy=None):
    from layer_util import f64
    return layer.head_norm(f64(host[which]), f64(host["w" + which]), norm=norm, eps=float(np.float32(1e-5)),
                           scale=float(np.float32(0.37)) if which == "q" else 1.0, cos=f64(host["cos"]),
                           sin=f64(host["sin"]), positions=None if host["pos"] is None else host["pos"].numpy(),
                           interleaved=interleaved, dy=dy)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("norm,interleaved", [("rms", False), ("l2", True)])
@pytest.mark.parametrize("case", QK, ids=lambda c: "-".join(map(str, c)))
def test_qk_norm(case, norm, interleaved, dt):
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, f64
    host, on = _qk_case(case, dt, 11, fuse=case[1] % 2 == 1)
    print(f"qk norm {case} {dt} {norm} interleaved={interleaved}", flush=True)
    kw = _kw(on, norm, interleaved)
    qo, ko = gdn.gdn_qk_norm_fwd(on["q"], on["k"], on["wq"], on["wk"], **kw)
    g = gdn.gdn_qk_norm_bwd(on["q"], on["k"], on["wq"], on["wk"], dq_out=on["dq"], dk_out=on["dk"], **kw)
    for which, out in (("q", qo), ("k", ko)):
        y, dx, dw = _want(host, which, norm, interleaved, dy=f64(host["d" + which]))
        check(out, y, which)
        check(g["d" + which], dx, "d" + which)
        check(g["dw" + which], dw, "dw" + which)


def test_qk_norm_without_weights_positions_or_upstream_in_bf16():
    """No weights: ones; no positions: 0 .. T-1; upstream gradients in float32."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, f64
    host, on = _qk_case((2, 33, 4, 2, 64, 32), "bf16", 12, fuse=False)
    host["pos"] = on["pos"] = None
    kw = _kw(on, "rms", False)
    qo, ko = gdn.gdn_qk_norm_fwd(on["q"], on["k"], **kw)
    g = gdn.gdn_qk_norm_bwd(on["q"], on["k"], dq_out=on["dq"].float(), dk_out=on["dk"].float(), **kw)
    assert sorted(g) == ["dk", "dq"]
    host["wq"] = host["wk"] = None
    for which, out in (("q", qo), ("k", ko)):
        y, dx, _ = _want(host, which, "rms", False, dy=f64(host["d" + which]))
        check(out, y, which)
        check(g["d" + which], dx, "d" + which)


@pytest.mark.parametrize("B,T,Hq,Hk,d", [(7, 1, 1, 1, 16), (300, 2, 1, 1, 16), (90, 3, 2, 1, 16), (50, 7, 1, 1, 32),
                                          (3, 129, 1, 1, 16), (2, 130, 5, 2, 16), (2, 999, 16, 8, 64), (40, 300, 3, 1, 16)])
def test_qk_norm_default_positions_are_those_of_each_sequence(B, T, Hq, Hk, d):
    """No positions: 0 .. T-1 in every sequence, bit for bit, where a step of the walk over the
    rows is many sequences, less than one, or a token's heads; several steps a block."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    _, on = _qk_case((B, T, Hq, Hk, d, 16), "f32", 18, fuse=False)
    kw = _kw(on, "rms", False)
    run = lambda: gdn.gdn_qk_norm_fwd(on["q"], on["k"], on["wq"], on["wk"], **kw) + tuple(  # noqa: E731
        gdn.gdn_qk_norm_bwd(on["q"], on["k"], on["wq"], on["wk"], dq_out=on["dq"], dk_out=on["dk"], **kw).values())
    kw["positions"] = torch.arange(T, dtype=torch.int32, device=dev()).expand(B, T).contiguous()
    want = run()
    kw["positions"] = None
    for x, y in zip(run(), want):
        assert torch.equal(x, y)


def test_qk_norm_in_place_equals_out_of_place():
    import gated_delta_rule_69_amd as gdn
    _, on = _qk_case((2, 41, 3, 2, 128, 128), "bf16", 13, fuse=False)
    kw = _kw(on, "rms", False)
    qo, ko = gdn.gdn_qk_norm_fwd(on["q"], on["k"], on["wq"], on["wk"], **kw)
    q, k = on["q"].clone(), on["k"].clone()
    q2, k2 = gdn.gdn_qk_norm_fwd(q, k, on["wq"], on["wk"], q_out=q, k_out=k, **kw)
    assert q2 is q and k2 is k
    assert torch.equal(qo, q) and torch.equal(ko, k)


def test_qk_norm_positions_outside_the_table_give_nan_rows():
    import gated_delta_rule_69_amd as gdn
    host, on = _qk_case((1, 6, 2, 1, 32, 16), "f32", 14, fuse=False)
    P = on["cos"].shape[0]
    kw = _kw(on, "rms", False)
    good, _ = gdn.gdn_qk_norm_fwd(on["q"], on["k"], on["wq"], on["wk"], **kw)
    bad = on["pos"].clone()
    bad[0, 1], bad[0, 4] = -1, P
    kw["positions"] = bad
    qo, ko = gdn.gdn_qk_norm_fwd(on["q"], on["k"], on["wq"], on["wk"], **kw)
    for t in (1, 4):
        assert torch.isnan(qo[0, t, :, :16]).all() and torch.isnan(ko[0, t, :, :16]).all()
    keep = [0, 2, 3, 5]
    assert torch.equal(qo[:, keep], good[:, keep])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,interleaved", [(32, 16, False), (64, 8, True), (128, 64, False), (128, 128, True)])
def test_qk_norm_positions_outside_the_table_are_nan_in_every_channel(d, rot, interleaved, dt):
    """Rotated channels or not: the whole row of the output and of its gradient, and the sums
    for the weights, which take every row in. Other rows keep their bits."""
    import gated_delta_rule_69_amd as gdn
    host, on = _qk_case((2, 7, 3, 2, d, rot), dt, 17, fuse=True)
    P = on["cos"].shape[0]
    kw = _kw(on, "l2", interleaved)
    run = lambda: gdn.gdn_qk_norm_fwd(on["q"], on["k"], on["wq"], on["wk"], **kw) + tuple(  # noqa: E731
        gdn.gdn_qk_norm_bwd(on["q"], on["k"], on["wq"], on["wk"], dq_out=on["dq"], dk_out=on["dk"], **kw)[n]
        for n in ("dq", "dk", "dwq", "dwk"))
    good = run()
    assert all(torch.isfinite(x).all() for x in good)
    bad = on["pos"].clone()
    bad[0, 1], bad[0, 6], bad[1, 3] = -1, P, 2 ** 31 - 1
    kw["positions"] = bad
    got = run()
    out = torch.zeros((2, 7), dtype=torch.bool)
    out[0, 1] = out[0, 6] = out[1, 3] = True
    for x, y in zip(got[:4], good[:4]):
        assert torch.isnan(x.cpu()[out]).all()
        assert torch.equal(x.cpu()[~out], y.cpu()[~out])
    for x in got[4:]:
        assert torch.isnan(x).all()


def test_qk_norm_zero_rows_and_many_rows():
    """Rows of zeros stay zero under eps; a launch of many blocks touches every row."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, dev, f64
    gen = torch.Generator().manual_seed(15)
    q = torch.randn((2, 5000, 3, 16), generator=gen).to(torch.bfloat16)
    q[0, 17] = 0
    k = torch.randn((2, 5000, 1, 16), generator=gen).to(torch.bfloat16)
    qo, ko = gdn.gdn_qk_norm_fwd(q.to(dev()), k.to(dev()), norm="l2")
    assert (qo[0, 17] == 0).all()
    check(qo, layer.head_norm(f64(q), norm="l2"), "q")
    check(ko, layer.head_norm(f64(k), norm="l2"), "k")
    dq = torch.randn(q.shape, generator=gen).to(torch.bfloat16)
    dk = torch.randn(k.shape, generator=gen).to(torch.bfloat16)
    one = torch.ones(16, device=dev())
    g = gdn.gdn_qk_norm_bwd(q.to(dev()), k.to(dev()), one, one, dq_out=dq.to(dev()), dk_out=dk.to(dev()))
    for n, x, d in (("q", q, dq), ("k", k, dk)):
        _, dx, dw = layer.head_norm(f64(x), dy=f64(d))
        check(g["d" + n], dx, "d" + n)
        check(g["dw" + n], dw, "dw" + n)


GATED = [(1, 1, 1, 16), (2, 37, 3, 16), (3, 19, 5, 64), (1, 130, 2, 32), (2, 700, 16, 128)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
@pytest.mark.parametrize("case", GATED, ids=lambda c: "-".join(map(str, c)))
def test_gated_norm(case, activation, dt):
    import gated_delta_rule_69_amd as gdn
    from layer_util import DTYPES, check, dev, f64, fused, rand
    B, T, H, d = case
    gen = torch.Generator().manual_seed(21)
    dtype = DTYPES[dt]
    x, z, dy = (rand(gen, case, dtype, s) for s in (0.5, 2.0, 1.0))
    w = 1 + rand(gen, (d,), torch.float32, 0.2)
    xd, zd = fused([x, z]) if T % 2 else (x.to(dev()), z.to(dev()))
    print(f"gated norm {case} {dt} {activation}", flush=True)
    y = gdn.gdn_gated_norm_fwd(xd, zd, w.to(dev()), activation=activation, eps=1e-5)
    g = gdn.gdn_gated_norm_bwd(xd, zd, w.to(dev()), d_out=dy.to(dev()), activation=activation, eps=1e-5)
    want = layer.gated_norm(f64(x), f64(z), f64(w), eps=float(np.float32(1e-5)), activation=activation, dy=f64(dy))
    for got, ref, name in zip((y, g["dx"], g["dgate"], g["dw"]), want, ("y", "dx", "dgate", "dw")):
        check(got, ref, name)


def test_gated_norm_extremes_in_place_and_no_weight():
    """Gates far out saturate without NaN; the output may be x itself; no weight: ones."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, dev, f64, rand
    gen = torch.Generator().manual_seed(22)
    x = rand(gen, (1, 9, 2, 32), torch.float32)
    z = rand(gen, (1, 9, 2, 32), torch.float32)
    z[0, 3], z[0, 4] = -120.0, 120.0
    y = gdn.gdn_gated_norm_fwd(x.to(dev()), z.to(dev()))
    check(y, layer.gated_norm(f64(x), f64(z)), "y")
    xi = x.to(dev())
    assert gdn.gdn_gated_norm_fwd(xi, z.to(dev()), out=xi) is xi and torch.equal(xi, y)
    g = gdn.gdn_gated_norm_bwd(x.to(dev()), z.to(dev()), d_out=torch.ones_like(y))
    assert sorted(g) == ["dgate", "dx"] and all(torch.isfinite(t).all() for t in g.values())


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
def test_gated_norm_float32_gate_far_out(activation):
    """Every output to a few float32 steps, nearly closed gates too: rows of +-1 have r = 1, so
    y is +-act(z). e^-z and the reciprocal are within a step of 2^-23 each, 1 + e^-z, z times
    the sigmoid and the three products within half of one, r within a step: 5.5 steps."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev, f64
    z = torch.linspace(-80, 30, 8 * 128).reshape(1, 8, 1, 128)
    x = torch.where(torch.arange(128) % 3 == 0, -1.0, 1.0).expand(z.shape).contiguous()
    y = f64(gdn.gdn_gated_norm_fwd(x.to(dev()), z.to(dev()), eps=0.0, activation=activation))
    want = layer.gated_norm(f64(x), f64(z), eps=0.0, activation=activation)
    assert (abs(y - want) <= 5.5 * 2.0 ** -23 * abs(want)).all(), float((abs(y - want) / abs(want)).max() * 2 ** 23)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
def test_gated_norm_gradient_of_a_gate_far_out(activation, dt):
    """Every element of dgate, gates wide open too, where 1 - sigmoid is far under a step of 1.
    Rows of +-1 with upstream 1 have r = 1, so dgate is +-act'(z). In steps of 2^-23, with n
    those of e = e^-|z| (1 for float32; 1 + |z| / 2 for bf16, whose exponent is rounded first):
    1 / (1 + e) takes n / 2 + 1.5 (half a step of the sum, one of the reciprocal), e / (1 + e)
    n + 2. Sigmoid: their product and its half step, 1.5 n + 4. SiLU, s (1 + z rest): n + 2.5
    of z rest, half a step of the sum, n + 2.5 of the product with s. Then the output's own half
    step, 2^-8 or 2^-24 of the value."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import DTYPES, dev, f64
    z = torch.linspace(-80, 80, 16 * 128).reshape(1, 16, 1, 128).to(DTYPES[dt])
    x = torch.where(torch.arange(128) % 3 == 0, -1.0, 1.0).expand(z.shape).to(z.dtype).contiguous()
    got = gdn.gdn_gated_norm_bwd(x.to(dev()), z.to(dev()), d_out=torch.ones_like(x).to(dev()), eps=0.0, activation=activation)
    zz = f64(z)
    s, rest = 1 / (1 + np.exp(-zz)), 1 / (1 + np.exp(zz))
    # written out: the oracle's 1 - s is 0 in 64 bits from z = 37 on
    want = np.sign(f64(x)) * (s * rest if activation == "sigmoid" else s * (1 + zz * rest))
    n = 1.0 if dt == "f32" else 1 + abs(zz) / 2
    steps = (1.5 * n + 4) * abs(want) if activation == "sigmoid" else s * abs(zz) * rest * (n + 2.5) + (n + 3) * abs(want)
    bound = steps * 2.0 ** -23 + abs(want) * (2.0 ** -8 if dt == "bf16" else 2.0 ** -24)
    off = abs(f64(got["dgate"]) - want)
    assert (off <= bound).all(), (float(zz.flatten()[(off / bound).argmax()]), float((off / bound).max()))


def test_norms_of_no_tokens():
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    x = torch.empty((2, 0, 3, 32), device=dev())
    w = torch.ones(32, device=dev())
    assert gdn.gdn_gated_norm_fwd(x, x, w).shape == x.shape
    assert torch.equal(gdn.gdn_gated_norm_bwd(x, x, w, d_out=x)["dw"], torch.zeros(32, device=dev()))
    q, k = gdn.gdn_qk_norm_fwd(x, x, w, w)
    assert q.shape == k.shape == x.shape
    g = gdn.gdn_qk_norm_bwd(x, x, w, w, dq_out=x, dk_out=x)
    assert torch.equal(g["dwq"], torch.zeros(32, device=dev())) and torch.equal(g["dwk"], g["dwq"])
