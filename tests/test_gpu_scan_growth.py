"""The gated recurrence's log gate with f of both signs: decays above 1, next to decays that take what
they grew away again.

Errors are held against the same recurrence of magnitudes, |h| <= M_t = a M_{t-1} + |b| (and the
gradients' likewise), which is what roundings of the terms add up to. Float32: a value passes at most eight
tokens one by one (an exponential to 2^-23 and a rounding each), six joins and, for every 256 tokens,
one of a state, each some 2^-22: under 1e-5 for the lengths here. bf16 has exponents to |f| 2^-24 more,
under 2e-5 with |f| <= 4, and rounds once to half a step, 2^-8 of the value. df is the product of two such
values, and is held to twice as much."""
import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu

INF = float("inf")


def _near(got, want, size, name):
    from layer_util import f64
    bf16 = got.dtype == torch.bfloat16
    e, most = np.abs(f64(got) - want), (2.0 ** -8 * np.abs(want) + 2e-5 * size if bf16 else 1e-5 * size)
    assert np.isfinite(f64(got)).all(), f"{name}: not finite"
    worst = np.unravel_index(np.argmax(e - most), e.shape)
    assert (e <= most + 1e-37).all(), f"{name} at {worst}: {f64(got)[worst]} for {want[worst]}, off by {e[worst]:.2e} of at most {most[worst]:.2e}"


def _compare(x, f, i, h0, d_h, dh_final, lens=None, low=0.0):
    import gated_delta_rule_69_amd as gdn
    from block_util import lengths
    from layer_util import dev, f64
    up = lambda t: None if t is None else t.to(dev())  # noqa: E731
    kw = dict(gate="log", seq_lens=lengths(lens))
    host = [f64(t) for t in (x, f, i)]
    size = lambda t: None if t is None else np.abs(f64(t))  # noqa: E731
    sizes = [size(x), host[1], host[2]]
    want, end = block.scan_forward(*host, gate="log", h0=f64(h0), lens=lens)
    big, big_end = block.scan_forward(*sizes, gate="log", h0=size(h0), lens=lens)
    grads = block.scan_backward(*host, gate="log", d_h=f64(d_h), h0=f64(h0), dh_final=f64(dh_final), lens=lens)
    bounds = block.scan_backward(*sizes, gate="log", d_h=size(d_h), h0=size(h0), dh_final=size(dh_final), lens=lens)
    got, got_end, marks = gdn.gdn_gated_scan_fwd(up(x), up(f), up(i), h0=up(h0), want_checkpoints=True, **kw)
    _near(got, want, big, "h")
    _near(got_end, end, big_end, "h_final")
    for ck in (marks, None):
        g = gdn.gdn_gated_scan_bwd(up(x), up(f), up(i), d_h=up(d_h), h0=up(h0), dh_final=up(dh_final), checkpoints=ck, **kw)
        for n, t in g.items():
            _near(t, grads[n], bounds[n] * 2.0 + low / 1e-5 if n == "df" else bounds[n], n)
    state = up(h0).clone()
    one = gdn.gdn_gated_scan_step(up(x), up(f), up(i), state=state, **kw)
    # one by one: each token rounds, an exponential to 2^-23 and a sum, on top of the above
    each = x.shape[1] * 2.0 ** -22
    _near(one, want, big * (1 + each / 1e-5), "step h")
    _near(state, end, big_end * (1 + each / 1e-5), "step state")


@pytest.mark.parametrize("igate", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,spread,lens", [
    (1, 40, 8, 1.0, None), (2, 200, 24, 1.0, [200, 131]), (3, 300, 40, 0.8, None), (1, 700, 136, 0.6, None),
    (260, 600, 8, 0.5, None),              # one segment of several tiles
    (2, 2500, 40, 0.3, [2500, 1203]), (1, 5000, 16, 0.2, None)])
def test_growth_and_decay_mixed(B, T, C, spread, lens, dt, igate):
    from block_util import spoil
    from layer_util import DTYPES, rand
    print(f"growth {B} {T} {C} {dt} igate={igate}", flush=True)
    gen, dtype = torch.Generator().manual_seed(T), DTYPES[dt]
    x, d_h = (spoil(rand(gen, (B, T, C), dtype), lens) for _ in range(2))
    f = spoil(rand(gen, (B, T, C), dtype, spread), lens)
    i = spoil(rand(gen, (B, T, C), dtype), lens) if igate else None
    _compare(x, f, i, rand(gen, (B, C), torch.float32), d_h, rand(gen, (B, C), torch.float32), lens)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("each,by,T,h0", [(128, 0.125, 256, 1.0), (16, 1.0, 256, 1.0), (4, 3.0, 256, 1.0), (4, 4.0, 256, 1.0),
                                          (8, 4.0, 4096, 1.0), (64, 1.0, 4096, 1e-20), (128, 1.0, 2048, 1e-30), (16, -4.0, 1024, 1e20)])
def test_growth_taken_away_again_leaves_the_state(each, by, T, h0, dt):
    """A state that grows for some tokens and decays for as many, over and over, ends as it began."""
    from layer_util import DTYPES
    C, dtype = 8, DTYPES[dt]
    f = torch.where((torch.arange(T) // each) % 2 == 0, by, -by)[None, :, None].expand(1, T, C).to(dtype).contiguous()
    x = torch.zeros((1, T, C), dtype=dtype)
    h0 = torch.full((1, C), h0)
    _compare(x, f, None, h0, x, 1e-4 / h0)


@pytest.mark.parametrize("T,h0", [(1000, 0.0), (5000, 0.0), (80, 1.0)])
def test_growth_of_an_empty_state(T, h0):
    """What has grown e^T times is still 0 if it was; and a state may grow to the end of float32."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    for dtype in (torch.float32, torch.bfloat16):
        x, f = torch.zeros((1, T, 16), dtype=dtype, device=dev()), torch.ones((1, T, 16), dtype=dtype, device=dev())
        h, end = gdn.gdn_gated_scan_fwd(x, f, gate="log", h0=torch.full((1, 16), h0, device=dev()))
        g = gdn.gdn_gated_scan_bwd(x, f, gate="log", d_h=x, dh_final=torch.full((1, 16), h0, device=dev()))
        want = h0 * float(np.exp(float(T))) if h0 else 0.0
        for t in (end, g["dh0"]):
            assert torch.isfinite(t).all() and ((t - want).abs() <= 1e-5 * want).all()
        assert (g["dx"][:, 0] == 0).all() if h0 == 0 else torch.isfinite(g["dx"]).all()


@pytest.mark.parametrize("C", [16, 2048])
@pytest.mark.parametrize("first", [80.0, -110.0])
def test_growth_before_what_would_leave_nothing(first, C):
    """A stretch whose decays alone are under 2^-149, in one segment with a stretch that grew the state
    before it, or grows it after: nothing of either is left out. Both directions."""
    T, a, b = 9000, 350, 1200
    f = torch.zeros((1, T, C))
    f[:, 30:a] = first / (a - 30)
    f[:, a:b] = (-30.0 - first) / (b - a)
    gen = torch.Generator().manual_seed(C)
    d_h = torch.randn((1, T, C), generator=gen) * 1e-20
    h0 = torch.full((1, C), 1.0 if first > 0 else 1e20)
    _compare(torch.randn((1, T, C), generator=gen) * 1e-20, f, None, h0, d_h, torch.ones((1, C)))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_growth_after_a_reset(dt):
    """f = -Inf empties a state, whatever grew it before or grows it after."""
    from layer_util import DTYPES
    gen, dtype = torch.Generator().manual_seed(3), DTYPES[dt]
    B, T, C = 2, 700, 24
    f = torch.randn((B, T, C), generator=gen) * 0.5
    f[:, 100], f[0, 101], f[1, 300:303], f[:, 690] = -INF, -INF, -INF, -INF
    x, d_h = (torch.randn((B, T, C), generator=gen).to(dtype) for _ in range(2))
    _compare(x, f.to(dtype), None, torch.randn((B, C), generator=gen), d_h, torch.randn((B, C), generator=gen))


@pytest.mark.parametrize("f", [-0.1343, -0.09, -0.05, 0.0, -3.0])
@pytest.mark.parametrize("T", [40, 2000])
def test_decay_from_the_end_of_float32(T, f):
    """The largest states, whose decays have any fraction of a power of two.

    df = l a h, and where one of h and l falls below float32's normal range each of its tokens rounds to
    half of 2^-149, T of them at most (what they decay by since only takes from that); the other factor is up
    to 3.3e38. So df is off by T 2^-150 3.3e38 on top: l = 1e-37 e^-12 has ten bits, e^-24 of it none."""
    x = torch.zeros((1, T, 16))
    h0 = torch.full((1, 16), 3.3e38)
    low = T * 2.0 ** -150 * 3.3e38
    _compare(x, torch.full((1, T, 16), f), None, h0, x, torch.full((1, 16), 1e-37), low=low)
    _compare(x, torch.full((1, T, 16), f), None, torch.ones((1, 16)), x, h0, low=low)


@pytest.mark.parametrize("gate", ["log", "sigmoid", "power"])
@pytest.mark.parametrize("n,value", [("x", float("nan")), ("x", INF), ("f", float("nan")), ("i", float("nan"))])
@pytest.mark.parametrize("T,at", [(12, 3), (300, 37), (4000, 700)])
def test_nan_and_inf_stay_in_their_channel_for_every_gate(T, at, n, value, gate):
    """From its row on, under decays that leave weights over 2^-127; nothing before and beside it changes, and
    in the gradients nothing beside its channel."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    gen = torch.Generator().manual_seed(T)
    B, C = 2, 24
    t = {k: torch.randn((B, T, C), generator=gen).to(dev()) for k in ("x", "f", "i", "d_h")}
    if gate != "power":
        t["f"] = t["f"] * 0.01 if gate == "log" else t["f"].abs() + 4.5
    decay = torch.full((C,), 0.01, device=dev()) if gate == "power" else None

    def run():
        a = (t["x"], t["f"], t["i"])
        kw = dict(gate=gate, decay=decay)
        return (gdn.gdn_gated_scan_fwd(*a, **kw)[0], gdn.gdn_gated_scan_bwd(*a, d_h=t["d_h"], **kw),
                gdn.gdn_gated_scan_step(*a, state=torch.zeros((B, C), device=dev()), **kw))

    clean = run()
    t[n][1, at, 5] = value
    got = run()
    for h, want in ((got[0], clean[0]), (got[2], clean[2])):
        assert not torch.isfinite(h[1, at:, 5]).any()
        h[1, at:, 5] = want[1, at:, 5]
        assert torch.equal(h, want)
    for k, g in got[1].items():
        want = clean[1][k]
        (g[5:6] if g.dim() == 1 else g[1, ..., 5]).copy_(want[5:6] if g.dim() == 1 else want[1, ..., 5])
        assert torch.equal(g, want), k
    if n == "f":   # l runs through a from the row on backwards
        g = gdn.gdn_gated_scan_bwd(t["x"], t["f"], t["i"], d_h=t["d_h"], gate=gate, decay=decay)
        assert not torch.isfinite(g["dx"][1, :at, 5]).any() and not torch.isfinite(g["dh0"][1, 5])
