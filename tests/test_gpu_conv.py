"""The short causal convolution against its float64 definition (oracle.block)."""
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu

CASES = [(1, 1, 8, None), (2, 2, 24, None), (3, 3, 16, [3, 0, 1]), (1, 5, 264, None), (2, 31, 8, [2, 31]), (1, 64, 40, None),
         (4, 65, 520, [65, 1, 33, 64]), (2, 257, 136, [-1, 300]), (1, 1000, 24, None), (2, 2049, 16, [2049, 2048]),
         (1030, 9, 8, None), (1030, 33, 8, None)]   # many sequences: up to 32 tokens one by one


def _case(B, T, C, W, dt, seed, lens=None, bias=True):
    from block_util import spoil
    from layer_util import DTYPES, rand
    gen = torch.Generator().manual_seed(seed)
    dtype = DTYPES[dt]
    return dict(x=spoil(rand(gen, (B, T, C), dtype), lens), w=rand(gen, (C, W), torch.float32, W ** -0.5),
                bias=rand(gen, (C,), torch.float32, 0.3) if bias else None, s0=rand(gen, (B, W - 1, C), dtype),
                d_y=spoil(rand(gen, (B, T, C), dtype), lens), ds_final=rand(gen, (B, W - 1, C), dtype))


@pytest.mark.parametrize("activation", ["silu", None])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:3])))
def test_conv(case, dt, W, activation):
    import gated_delta_rule_69_amd as gdn
    from block_util import host, lengths, on
    from layer_util import check, dev
    B, T, C, lens = case
    print(f"conv {case} {dt} W={W} {activation}", flush=True)
    c = _case(B, T, C, W, dt, seed=T + W, lens=lens, bias=T % 2 == 1)
    d, h = {k: None if v is None else v.to(dev()) for k, v in c.items()}, host(c)
    d["x"] = on(c["x"], wide=C % 16 == 8)
    s0, hs0 = (d["s0"], h["s0"]) if T % 3 else (None, None)
    up, hup = (d["ds_final"], h["ds_final"]) if T % 3 else (None, None)
    kw = dict(activation=activation, seq_lens=lengths(lens))
    want, want_end = block.conv_forward(h["x"], h["w"], h["bias"], activation=activation, s0=hs0, lens=lens)
    y, end = gdn.gdn_short_conv_fwd(d["x"], d["w"], d["bias"], s0=s0, **kw)
    check(y, want, "y")
    check(end, want_end, "s_final")
    given = torch.full_like(y, 7.0)
    gdn.gdn_short_conv_fwd(d["x"], d["w"], d["bias"], s0=s0, y=given, want_state=False, **kw)
    for b in range(B):
        n = T if lens is None else min(max(lens[b], 0), T)
        assert torch.equal(given[b, :n], y[b, :n]) and (given[b, n:] == 7.0).all() and (y[b, n:] == 0).all()
    state = d["s0"].clone() if s0 is not None else torch.zeros_like(d["s0"])
    one = gdn.gdn_short_conv_step(d["x"], d["w"], d["bias"], state=state, **kw)
    assert torch.equal(one, y) and torch.equal(state, end)
    ref = block.conv_backward(h["x"], h["w"], h["bias"], d_y=h["d_y"], activation=activation, s0=hs0, ds_final=hup, lens=lens)
    g = gdn.gdn_short_conv_bwd(d["x"], d["w"], d["bias"], d_y=d["d_y"], s0=s0, ds_final=up, **kw)
    assert sorted(g) == (["dbias"] if c["bias"] is not None else []) + ["ds0", "dw", "dx"]
    for n, t in g.items():
        check(t, ref[n], n)
    for b in range(B if lens else 0):
        assert (g["dx"][b, max(lens[b], 0):] == 0).all()


@pytest.mark.parametrize("W", [2, 4])
def test_conv_prompt_then_tokens_is_the_whole(W):
    """Bit for bit: every token's sum has one order."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    d = {k: v.to(dev()) for k, v in _case(3, 90, 72, W, "bf16", 3).items()}
    whole, end = gdn.gdn_short_conv_fwd(d["x"], d["w"], d["bias"], s0=d["s0"])
    state = d["s0"].clone()
    rows = []
    for a, b in ((0, 1), (1, 2), (2, 60), (60, 61), (61, 90)):
        y, out = gdn.gdn_short_conv_fwd(d["x"][:, a:b].contiguous(), d["w"], d["bias"], s0=state, s_final=state)
        assert out is state
        rows.append(y)
    assert torch.equal(torch.cat(rows, 1), whole) and torch.equal(state, end)


def test_conv_nan_reaches_the_rows_that_read_it():
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    d = {k: v.to(dev()) for k, v in _case(2, 100, 16, 4, "f32", 4).items()}
    clean, _ = gdn.gdn_short_conv_fwd(d["x"], d["w"], d["bias"])
    d["x"][1, 37, 3] = float("nan")
    y, _ = gdn.gdn_short_conv_fwd(d["x"], d["w"], d["bias"])
    assert torch.isnan(y[1, 37:41, 3]).all()
    y[1, 37:41, 3] = clean[1, 37:41, 3]
    assert torch.equal(y, clean)


def test_conv_open_gates_and_large_sums():
    """silu of sums up to +-300: 0 and the sum itself, no overflow; its slope too."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, dev, f64
    x = torch.linspace(-300, 300, 64).reshape(1, 8, 8).contiguous()
    w = torch.zeros((8, 2))
    w[:, 1] = 1.0
    d_y = torch.ones_like(x)
    y, _ = gdn.gdn_short_conv_fwd(x.to(dev()), w.to(dev()))
    want, _ = block.conv_forward(f64(x), f64(w))
    check(y, want, "y")
    g = gdn.gdn_short_conv_bwd(x.to(dev()), w.to(dev()), d_y=d_y.to(dev()))
    ref = block.conv_backward(f64(x), f64(w), d_y=f64(d_y))
    for n in g:
        check(g[n], ref[n], n)


def test_conv_streams_graph_and_empty():
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    d = {k: v.to(dev()) for k, v in _case(2, 700, 136, 4, "bf16", 5).items()}

    def work(**k):
        y, end = gdn.gdn_short_conv_fwd(d["x"], d["w"], d["bias"], s0=d["s0"], **k)
        g = gdn.gdn_short_conv_bwd(d["x"], d["w"], d["bias"], d_y=d["d_y"], s0=d["s0"], ds_final=d["ds_final"], **k)
        return [y, end, *g.values()]

    want = work()
    torch.cuda.synchronize()
    both = [work(stream=torch.cuda.Stream(device=dev())) for _ in range(2)]
    torch.cuda.synchronize()
    for other in both:
        for x, y in zip(want, other):
            assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for _ in range(4):
        d["x"].mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, work()):
            assert torch.equal(x, y)
    none = d["x"][:, :0].contiguous()
    y, end = gdn.gdn_short_conv_fwd(none, d["w"], s0=d["s0"])
    assert y.shape == none.shape and torch.equal(end, d["s0"])
    g = gdn.gdn_short_conv_bwd(none, d["w"], d["bias"], d_y=none, ds_final=d["ds_final"])
    assert torch.equal(g["ds0"], d["ds_final"]) and (g["dw"] == 0).all() and (g["dbias"] == 0).all()


@pytest.mark.parametrize("B,T,C", [(4096, 3, 8), (1, 5, 65536), (1, 40000, 8)])
def test_conv_wide_long_and_many(B, T, C):
    import gated_delta_rule_69_amd as gdn
    from block_util import host
    from layer_util import check, dev
    c = _case(B, T, C, 4, "bf16", 6)
    d, h = {k: v.to(dev()) for k, v in c.items()}, host(c)
    y, end = gdn.gdn_short_conv_fwd(d["x"], d["w"], d["bias"], s0=d["s0"])
    want, want_end = block.conv_forward(h["x"], h["w"], h["bias"], s0=h["s0"])
    check(y, want, "y")
    check(end, want_end, "s_final")


def test_conv_gradients_against_differences():
    """The kernels' own forward pass in float32: y is off by 2^-21 of its size, which at a step of
    2^-7 is 2^-15 of it in the quotient; checked to 1e-3 of the largest."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    d = {k: v.to(dev()) for k, v in _case(1, 20, 8, 4, "f32", 7).items()}

    def loss():
        y, end = gdn.gdn_short_conv_fwd(d["x"], d["w"], d["bias"], s0=d["s0"])
        return ((y.double() * d["d_y"].double()).sum() + (end.double() * d["ds_final"].double()).sum()).item()

    g = gdn.gdn_short_conv_bwd(d["x"], d["w"], d["bias"], d_y=d["d_y"], s0=d["s0"], ds_final=d["ds_final"])
    e = 2.0 ** -7
    for n in ("x", "w", "bias", "s0"):
        flat, grad = d[n].view(-1), g["d" + n].reshape(-1)
        for k in range(0, flat.numel(), max(1, flat.numel() // 9)):
            keep = flat[k].item()
            flat[k] = keep + e
            up = loss()
            flat[k] = keep - e
            down = loss()
            flat[k] = keep
            assert abs((up - down) / (2 * e) - grad[k].item()) < 1e-3 * grad.abs().max().item(), (n, k)
