"""The gated recurrence a channel against its float64 definition (oracle.block)."""
import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu

# B, T, C, lens
CASES = [
    (1, 1, 8, None), (2, 2, 16, None), (1, 7, 24, None), (3, 8, 40, [8, 0, 3]), (1, 9, 8, None), (2, 63, 24, None),
    (2, 64, 16, None), (1, 65, 136, None), (2, 255, 32, [255, 64]), (1, 256, 8, None), (4, 257, 72, [257, 0, 1, 256]),
    (2, 511, 24, [-3, 900]), (1, 1025, 264, None), (2, 2500, 40, [2500, 1200]), (1, 5000, 16, None),
    (40, 30, 512, None), (40, 35, 512, None),     # more than 256 workgroups: up to 32 tokens one by one
]


def _device(case, wide):
    from block_util import dev, on
    return {k: None if v is None else on(v, wide and k in ("x", "f", "i")) if v.dim() == 3 else v.to(dev()) for k, v in case.items()}


@pytest.mark.parametrize("igate", [False, True])
@pytest.mark.parametrize("gate", ["log", "sigmoid", "power"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:3])))
def test_scan(case, dt, gate, igate):
    import gated_delta_rule_69_amd as gdn
    from block_util import host, lengths, scan_case
    from gated_delta_rule_69_amd._block import SCAN_SPAN as SPAN
    from layer_util import check, f64
    B, T, C, lens = case
    print(f"scan {case} {dt} {gate} igate={igate}", flush=True)
    c = scan_case(B, T, C, dt, gate, igate, seed=T, h0=T % 2 == 1, lens=lens)
    d, h = _device(c, wide=C % 16 == 8), host(c)
    kw, ref = dict(gate=gate, decay=d["decay"]), dict(gate=gate, decay=h["decay"], lens=lens)
    want, want_end = block.scan_forward(h["x"], h["f"], h["i"], h0=h["h0"], **ref)
    kw["seq_lens"] = lengths(lens)
    out, end, marks = gdn.gdn_gated_scan_fwd(d["x"], d["f"], d["i"], h0=d["h0"], want_checkpoints=True, **kw)
    check(out, want, "h")
    check(end, want_end, "h_final")
    # rows behind the lengths: zero if allocated, as they were if given
    given = torch.full_like(out, 7.0)
    again, end2 = gdn.gdn_gated_scan_fwd(d["x"], d["f"], d["i"], h0=d["h0"], h=given, **kw)
    assert again is given and torch.equal(end2, end)
    for b in range(B):
        n = T if lens is None else min(max(lens[b], 0), T)
        assert torch.equal(given[b, :n], out[b, :n]) and (given[b, n:] == 7.0).all() and (out[b, n:] == 0).all()
        for j in range(-(-n // SPAN)):
            before = want[b, SPAN * j - 1] if j else (np.zeros(C) if h["h0"] is None else h["h0"][b])
            np.testing.assert_allclose(f64(marks[b, j]), before, rtol=0, atol=1e-5 * max(1, abs(want).max()))
    # gradients, with the checkpoints and without
    ref["h0"] = h["h0"]
    grads = block.scan_backward(h["x"], h["f"], h["i"], d_h=h["d_h"], dh_final=h["dh_final"], **ref)
    for ck in (marks, None):
        got = gdn.gdn_gated_scan_bwd(d["x"], d["f"], d["i"], d_h=d["d_h"], h0=d["h0"], dh_final=d["dh_final"], checkpoints=ck, **kw)
        assert sorted(got) == sorted(grads)
        for n, g in got.items():
            check(g, grads[n], n)
            if g.dim() == 3:
                for b in range(B if lens else 0):
                    assert (g[b, max(lens[b], 0):] == 0).all(), n
    # token by token
    state = d["h0"].clone() if d["h0"] is not None else torch.zeros((B, C), device=out.device)
    one = gdn.gdn_gated_scan_step(d["x"], d["f"], d["i"], state=state, **kw)
    check(one, want, "step h")
    check(state, want_end, "step state")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["log", "sigmoid", "power"])
def test_scan_prompt_then_tokens_is_the_whole(gate, dt):
    import gated_delta_rule_69_amd as gdn
    from block_util import host, scan_case
    from layer_util import check
    B, T, C = 3, 300, 48
    c = scan_case(B, T, C, dt, gate, True, seed=5)
    d, h = _device(c, wide=False), host(c)
    kw = dict(gate=gate, decay=d["decay"])
    want, want_end = block.scan_forward(h["x"], h["f"], h["i"], gate=gate, decay=h["decay"], h0=h["h0"])
    part = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    state = d["h0"].clone()
    rows = []
    o, end = gdn.gdn_gated_scan_fwd(*(part(d[n], 0, 290) for n in "xfi"), h0=state, h_final=state, **kw)
    assert end is state                                         # in place
    rows.append(o)
    for t in range(290, T):
        rows.append(gdn.gdn_gated_scan_step(*(part(d[n], t, t + 1) for n in "xfi"), state=state, **kw))
    check(torch.cat(rows, 1), want, "h")
    check(state, want_end, "state")


@pytest.mark.parametrize("T,B,C", [(70000, 1, 8), (40000, 2, 24)])
@pytest.mark.parametrize("gate", ["log", "sigmoid", "power"])
def test_scan_channels_that_keep_many_tokens(gate, T, B, C):
    """Decays within 1e-6 .. 1e-4 of 1, the same at every token: what a rounded decay would be off
    by must not add up. Float32 to 2e-5: ten times the roundings of a sum of 1e5 terms in a tree
    (17 levels of 2^-24, 1e-6), on top of gates that are off by 2^-22 of 1 - a (a few steps)."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev, f64
    gen = torch.Generator().manual_seed(3)
    keep = torch.logspace(-6, -4, C, dtype=torch.float64)
    x = (torch.randn((B, T, C), generator=gen, dtype=torch.float64) + 1).float()
    f = {"log": -keep, "sigmoid": torch.log((1 - keep) / keep),
         "power": torch.zeros(C, dtype=torch.float64)}[gate].float().expand(B, T, C).contiguous()
    decay = (2 * keep).float() if gate == "power" else None
    h0 = torch.ones((B, C))
    d_h = torch.randn((B, T, C), generator=gen) + 0.5
    up = lambda t: None if t is None else t.to(dev())  # noqa: E731
    h, end, marks = gdn.gdn_gated_scan_fwd(up(x), up(f), gate=gate, decay=up(decay), h0=up(h0), want_checkpoints=True)
    g = gdn.gdn_gated_scan_bwd(up(x), up(f), gate=gate, decay=up(decay), h0=up(h0), d_h=up(d_h), checkpoints=marks)
    xd, fd = f64(x), f64(f)
    a, m = block._gates(fd[0, 0], gate, None if decay is None else f64(decay))
    state, lam = f64(h0), np.zeros((B, C))
    want, back = np.zeros(xd.shape), np.zeros(xd.shape)
    for t in range(T):
        state = a * state + m * xd[:, t]
        want[:, t] = state
    for t in range(T - 1, -1, -1):
        lam = lam + f64(d_h)[:, t]
        back[:, t] = lam
        lam = a * lam
    for c in range(C):
        e = np.abs(f64(h)[..., c] - want[..., c]).max() / np.abs(want[..., c]).max()
        eb = np.abs(f64(g["dx"])[..., c] - back[..., c] * m[c]).max() / np.abs(back[..., c] * m[c]).max()
        assert e < 2e-5 and eb < 2e-5, (gate, c, e, eb)
    np.testing.assert_allclose(f64(g["dh0"]), lam, rtol=2e-5, atol=2e-5 * np.abs(lam).max())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_extreme_gates(dt):
    """Closed, open and saturated gates: a = 0 and a = 1 exactly, logits up to the infinities."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import DTYPES, check, dev, f64
    inf = float("inf")
    T, C = 200, 16
    gen = torch.Generator().manual_seed(9)
    x = torch.randn((1, T, C), generator=gen).to(DTYPES[dt])
    d_h = torch.randn((1, T, C), generator=gen).to(DTYPES[dt])
    for gate, values in (("log", [0.0, -inf, -300.0, -90.0, -1e-30, -1.0]), ("sigmoid", [inf, -inf, 300.0, -300.0, 90.0, -90.0, 20.0]),
                         ("power", [inf, -inf, 300.0, -300.0, 90.0, -90.0, 0.0])):
        pick = torch.randint(0, len(values), (1, T, C), generator=gen)
        f = torch.tensor(values)[pick].to(DTYPES[dt])
        decay = torch.tensor([0.0, 1e-30, 1e-6, 1.0, 50.0, 400.0, 3.0, 0.5] * 2) if gate == "power" else None
        dc = None if decay is None else decay.to(dev())
        h0 = torch.ones((1, C), device=dev())
        h, end = gdn.gdn_gated_scan_fwd(x.to(dev()), f.to(dev()), gate=gate, decay=dc, h0=h0)
        want, want_end = block.scan_forward(f64(x), f64(f), gate=gate, decay=None if decay is None else f64(decay), h0=f64(h0))
        check(h, want, f"{gate} h")
        check(end, want_end, f"{gate} end")
        g = gdn.gdn_gated_scan_bwd(x.to(dev()), f.to(dev()), gate=gate, decay=dc, h0=h0, d_h=d_h.to(dev()))
        ref = block.scan_backward(f64(x), f64(f), d_h=f64(d_h), gate=gate, decay=None if decay is None else f64(decay), h0=f64(h0))
        for n in ("dx", "dh0", "df"):
            check(g[n], ref[n], f"{gate} {n}")
        if gate == "power":
            ok = (decay > 1e-20).numpy()      # at decay 0 the slope of m has no limit
            check(g["ddecay"][torch.from_numpy(ok).to(dev())], ref["ddecay"][ok], "ddecay")


@pytest.mark.parametrize("slow", [False, True])
@pytest.mark.parametrize("T,B,C", [(9000, 1, 2048), (9000, 2, 256)])
def test_scan_long_segments(T, B, C, slow):
    """Segments of several tiles, whose totals stop where nothing before them is left: in no slice, or in
    those that hold one channel that forgets nothing. Both directions (C 2048 and 256: several tiles a
    segment forwards, and in the gradients)."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, dev, f64
    gen = torch.Generator().manual_seed(C)
    x, d_h = (torch.randn((B, T, C), generator=gen) for _ in range(2))
    f = -torch.rand((B, T, C), generator=gen) * 0.5
    if slow:
        f[:, :, 5::130] = -1e-4
    h0, up = (torch.randn((B, C), generator=gen) for _ in range(2))
    out, end = gdn.gdn_gated_scan_fwd(x.to(dev()), f.to(dev()), gate="log", h0=h0.to(dev()))
    g = gdn.gdn_gated_scan_bwd(x.to(dev()), f.to(dev()), gate="log", h0=h0.to(dev()), d_h=d_h.to(dev()), dh_final=up.to(dev()))
    want, want_end = block.scan_forward(f64(x), f64(f), gate="log", h0=f64(h0))
    ref = block.scan_backward(f64(x), f64(f), d_h=f64(d_h), gate="log", h0=f64(h0), dh_final=f64(up))
    check(out, want, "h")
    check(end, want_end, "end")
    for n in ("dx", "df", "dh0"):
        check(g[n], ref[n], n)
    inplace = h0.to(dev())
    again, same = gdn.gdn_gated_scan_fwd(x.to(dev()), f.to(dev()), gate="log", h0=inplace, h_final=inplace)
    assert same is inplace and torch.equal(same, end) and torch.equal(again, out)


def test_scan_jump_of_magnitude_leaves_later_rows_exact():
    """What decays away leaves nothing behind: rows after a reset keep their own relative accuracy
    next to values 1e12 larger before it."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev, f64
    T, C = 700, 8
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((1, T, C), generator=gen)
    f = torch.full((1, T, C), -0.05)
    x[:, :300] *= 1e12
    f[:, 300:330] = -3.0
    h, _ = gdn.gdn_gated_scan_fwd(x.to(dev()), f.to(dev()), gate="log")
    want, _ = block.scan_forward(f64(x), f64(f), gate="log")
    err = np.abs(f64(h) - want)[:, 340:]
    assert err.max() < 1e-5 * np.abs(want[:, 340:]).max()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,at", [(40, 3), (1100, 70), (5000, 600)])
def test_scan_nan_and_inf_stay_in_their_channel(T, at, value):
    import gated_delta_rule_69_amd as gdn
    from block_util import scan_case
    c = scan_case(2, T, 24, "f32", "sigmoid", False, seed=2)
    d = _device(c, wide=False)
    clean, clean_end = gdn.gdn_gated_scan_fwd(d["x"], d["f"], h0=d["h0"])
    d["x"][1, at, 5] = value
    h, end = gdn.gdn_gated_scan_fwd(d["x"], d["f"], h0=d["h0"])
    assert not torch.isfinite(h[1, at:, 5]).any() and not torch.isfinite(end[1, 5])
    h[1, at:, 5], end[1, 5] = clean[1, at:, 5], clean_end[1, 5]
    assert torch.equal(h, clean) and torch.equal(end, clean_end)


def test_scan_is_deterministic_and_independent_of_other_streams():
    import gated_delta_rule_69_amd as gdn
    from block_util import dev, scan_case
    c = scan_case(2, 3000, 72, "bf16", "power", True, seed=4)
    d = _device(c, wide=False)
    kw = dict(gate="power", decay=d["decay"], h0=d["h0"])
    run = lambda **k: list(gdn.gdn_gated_scan_fwd(d["x"], d["f"], d["i"], **kw, **k)) + list(  # noqa: E731
        gdn.gdn_gated_scan_bwd(d["x"], d["f"], d["i"], d_h=d["d_h"], dh_final=d["dh_final"], **kw, **k).values())
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=dev()) for _ in range(2)]
    got = [run(stream=s) for s in streams]
    torch.cuda.synchronize()
    for other in got + [run()]:
        for x, y in zip(want, other):
            assert torch.equal(x, y)


def test_scan_in_a_captured_graph():
    import gated_delta_rule_69_amd as gdn
    from block_util import dev, scan_case
    c = scan_case(2, 2100, 40, "bf16", "power", True, seed=6)
    d = _device(c, wide=False)
    kw = dict(gate="power", decay=d["decay"], h0=d["h0"])

    def work():
        h, end, marks = gdn.gdn_gated_scan_fwd(d["x"], d["f"], d["i"], want_checkpoints=True, **kw)
        g = gdn.gdn_gated_scan_bwd(d["x"], d["f"], d["i"], d_h=d["d_h"], checkpoints=marks, **kw)
        return [h, end, *g.values()]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for k in range(4):
        d["x"].mul_(0.5 + k), d["h0"].add_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, work()):
            assert torch.equal(x, y)


def test_scan_empty_batches_and_gradient_without_tokens():
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    x = torch.zeros((2, 0, 16), device=dev())
    h0 = torch.randn((2, 16), device=dev())
    h, end = gdn.gdn_gated_scan_fwd(x, x, h0=h0)
    assert h.shape == x.shape and torch.equal(end, h0)
    _, end = gdn.gdn_gated_scan_fwd(x, x)
    assert (end == 0).all()
    decay = torch.ones(16, device=dev())
    g = gdn.gdn_gated_scan_bwd(x, x, d_h=x, dh_final=h0, gate="power", decay=decay)
    assert torch.equal(g["dh0"], h0) and (g["ddecay"] == 0).all()
    state = h0.clone()
    gdn.gdn_gated_scan_step(x, x, state=state)
    assert torch.equal(state, h0)


def test_scan_rows_far_apart():
    """Offsets beyond 32 bits: a view whose tokens lie 2^22 elements apart, rows over 4 GiB from the
    first, and many sequences."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, dev, f64
    T, C, ld = 1100, 16, 1 << 21
    big = torch.zeros((T * ld,), dtype=torch.bfloat16, device=dev())
    view = big.as_strided((1, T, C), (T * ld, ld, 1), 8 * 1024)
    gen = torch.Generator().manual_seed(8)
    x = torch.randn((1, T, C), generator=gen).bfloat16()
    f = (torch.randn((1, T, C), generator=gen) + 2).bfloat16()
    view.copy_(x.to(dev()))
    h, end = gdn.gdn_gated_scan_fwd(view, f.to(dev()))
    want, want_end = block.scan_forward(f64(x), f64(f))
    check(h, want, "h")
    check(end, want_end, "end")
    d_h = torch.randn((1, T, C), generator=gen).bfloat16()
    g = gdn.gdn_gated_scan_bwd(view, f.to(dev()), d_h=d_h.to(dev()))
    ref = block.scan_backward(f64(x), f64(f), d_h=f64(d_h))
    for n in ("dx", "df", "dh0"):
        check(g[n], ref[n], n)
    one = gdn.gdn_short_conv_fwd(view, torch.ones((C, 3), device=dev()), activation=None)[0]
    check(one, block.conv_forward(f64(x), np.ones((C, 3)), activation=None)[0], "conv")
    del view, big


@pytest.mark.parametrize("C", [8, 40])
def test_scan_rows_at_odd_multiples_of_sixteen_bytes(C):
    import gated_delta_rule_69_amd as gdn
    from block_util import dev, host, scan_case
    from layer_util import check
    c = scan_case(2, 300, C, "f32", "sigmoid", True, seed=21)
    d, h = _device(c, wide=False), host(c)
    for n in "xfi":
        big = torch.full((2, 300, C + 4), float("nan"), device=dev())
        big[..., 4:] = d[n]
        d[n] = big[..., 4:]
    out, end = gdn.gdn_gated_scan_fwd(d["x"], d["f"], d["i"], h0=d["h0"])
    g = gdn.gdn_gated_scan_bwd(d["x"], d["f"], d["i"], h0=d["h0"], d_h=d["d_h"], dh_final=d["dh_final"])
    want, want_end = block.scan_forward(h["x"], h["f"], h["i"], h0=h["h0"])
    ref = block.scan_backward(h["x"], h["f"], h["i"], h0=h["h0"], d_h=h["d_h"], dh_final=h["dh_final"])
    check(out, want, "h")
    check(end, want_end, "end")
    for n, t in g.items():
        check(t, ref[n], n)


@pytest.mark.parametrize("B,C", [(4096, 8), (3, 16384), (1, 65536)])
def test_scan_wide_and_many(B, C):
    import gated_delta_rule_69_amd as gdn
    from block_util import host, scan_case
    from layer_util import check
    c = scan_case(B, 11, C, "bf16", "sigmoid", False, seed=B)
    d, h = _device(c, wide=False), host(c)
    out, end = gdn.gdn_gated_scan_fwd(d["x"], d["f"], h0=d["h0"])
    want, want_end = block.scan_forward(h["x"], h["f"], h0=h["h0"])
    check(out, want, "h")
    check(end, want_end, "end")


def test_scan_gradients_against_differences():
    """The kernels' own forward pass, by differences in float32 inputs: (L(x + e) - L(x - e)) / 2e of
    a loss summed in float64. h is off by 2^-22 of its size, so at e = 2^-6 the quotient is off by
    some 2^-16 of h a row times a row's share of the loss; checked to 2e-3 of the largest."""
    import gated_delta_rule_69_amd as gdn
    from block_util import scan_case
    c = scan_case(1, 70, 8, "f32", "power", True, seed=12)
    d = _device(c, wide=False)

    def loss():
        h, end = gdn.gdn_gated_scan_fwd(d["x"], d["f"], d["i"], gate="power", decay=d["decay"], h0=d["h0"])
        return ((h.double() * d["d_h"].double()).sum() + (end.double() * d["dh_final"].double()).sum()).item()

    g = gdn.gdn_gated_scan_bwd(d["x"], d["f"], d["i"], d_h=d["d_h"], gate="power", decay=d["decay"], h0=d["h0"], dh_final=d["dh_final"])
    e = 2.0 ** -6
    for n, t in (("dx", "x"), ("df", "f"), ("di", "i"), ("dh0", "h0"), ("ddecay", "decay")):
        flat, grad = d[t].view(-1), g[n].reshape(-1)
        for k in range(0, flat.numel(), max(1, flat.numel() // 9)):
            keep, step = flat[k].item(), e if t != "decay" else e * flat[k].item()
            flat[k] = keep + step
            up = loss()
            flat[k] = keep - step
            down = loss()
            flat[k] = keep
            assert abs((up - down) / (2 * step) - grad[k].item()) < 2e-3 * grad.abs().max().item(), (n, k)
