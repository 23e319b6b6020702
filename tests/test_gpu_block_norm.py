"""The norms around a block against their float64 definition (oracle.block)."""
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]   # of y, of the residual
# B, T, C
CASES = [(1, 1, 8), (2, 3, 24), (1, 7, 504), (2, 5, 512), (1, 4, 520), (3, 11, 2048), (1, 5, 2568), (1, 3, 8192), (2, 2, 8200),
         (1, 3, 16384), (1, 600, 64)]


def _case(B, T, C, types, seed):
    from layer_util import DTYPES, rand
    gen = torch.Generator().manual_seed(seed)
    dt, rt = (DTYPES[t] for t in types)
    row = lambda s=0.2, m=1.0: (m + rand(gen, (C,), torch.float32, s)).float()  # noqa: E731
    return dict(residual=rand(gen, (B, T, C), rt, 2.0), y=rand(gen, (B, T, C), dt), gate=rand(gen, (B, T, C), dt, 1.5),
                weight=row(), post_weight=row(), scale=row(0.3, 0.5), d_out=rand(gen, (B, T, C), dt),
                d_residual_out=rand(gen, (B, T, C), rt))


def _device(c, wide=False):
    from block_util import dev, on
    return {k: None if v is None else on(v, wide and k in ("residual", "y", "gate")) if v.dim() == 3 else v.to(dev())
            for k, v in c.items()}


UPS = ("d_out", "d_residual_out")
NAMES = dict(dr="residual", dy="y", dgate="gate", dw="weight", dw_post="post_weight", dscale="scale")


def _compare(c, wide, **kw):
    import gated_delta_rule_69_amd as gdn
    from block_util import host
    from layer_util import check
    d, h = _device(c, wide), host(c)
    ins = {k: v for k, v in d.items() if k not in UPS}
    ups = {k: d[k] for k in UPS}
    r, n = gdn.gdn_block_norm_fwd(**ins, **kw)
    g = gdn.gdn_block_norm_bwd(**ins, **ups, **kw)
    want_r, want_n, want = block.block_norm(**h, **kw)
    check(r, want_r, "residual_out")
    check(n, want_n, "out")
    assert sorted(g) == sorted(k for k, v in NAMES.items() if c[v] is not None)
    for k, t in g.items():
        check(t, want[k], k)
    return d, r, n


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_block_norm(case, types, post, activation):
    print(f"block norm {case} {types} post={post} {activation}", flush=True)
    c = _case(*case, types, seed=case[2])
    if not post:
        c["post_weight"] = None
    _compare(c, wide=case[2] % 16 == 8, post_norm=post, activation=activation, residual_scale=0.75, eps=1e-5)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("absent", [("gate",), ("scale",), ("weight",), ("post_weight",), ("gate", "scale", "weight", "post_weight"),
                                    ("d_out",), ("d_residual_out",)])
def test_block_norm_absent_inputs(absent, types):
    c = _case(2, 9, 264, types, seed=1)
    c.update({n: None for n in absent})
    _compare(c, wide=False, post_norm=True, activation="silu")


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("C,T", [(512, 2101), (1544, 1030), (4104, 519), (8200, 517)])
def test_block_norm_many_rows(C, T, types):
    """More rows than workgroups in the gradients: each walks several, the last fewer."""
    _compare(_case(1, T, C, types, seed=C), wide=False, post_norm=True, activation="silu")


@pytest.mark.parametrize("C", [8, 512, 2056, 8200])
def test_block_norm_rows_at_odd_multiples_of_sixteen_bytes(C):
    """Float32 rows that start sixteen bytes after a multiple of 32: views four channels into tensors of
    C + 4."""
    import gated_delta_rule_69_amd as gdn
    from block_util import host
    from layer_util import check, dev
    c = _case(2, 5, C, ("f32", "f32"), seed=9)
    d, h = _device(c), host(c)
    for n in ("residual", "y", "gate"):
        big = torch.full((2, 5, C + 4), float("nan"), device=dev())
        big[..., 4:] = d[n]
        d[n] = big[..., 4:]
        assert d[n].data_ptr() % 32 == 16
    ins, ups = {k: v for k, v in d.items() if k not in UPS}, {k: d[k] for k in UPS}
    r, n = gdn.gdn_block_norm_fwd(**ins, post_norm=True)
    g = gdn.gdn_block_norm_bwd(**ins, **ups, post_norm=True)
    want_r, want_n, want = block.block_norm(**h, post_norm=True)
    check(r, want_r, "residual_out")
    check(n, want_n, "out")
    for k, t in g.items():
        check(t, want[k], k)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_norm_before_a_first_block(types):
    """No output of a block yet: the norm of the residual alone."""
    import gated_delta_rule_69_amd as gdn
    from block_util import host
    from layer_util import DTYPES, check
    c = _case(2, 7, 136, types, seed=2)
    c.update(y=None, gate=None, scale=None, post_weight=None)
    d, h = _device(c), host(c)
    r, n = gdn.gdn_block_norm_fwd(d["residual"], weight=d["weight"], out_dtype=DTYPES[types[0]])
    want_r, want_n, want = block.block_norm(**h)
    assert torch.equal(r, d["residual"])
    check(n, want_n, "out")
    g = gdn.gdn_block_norm_bwd(d["residual"], weight=d["weight"], d_out=d["d_out"], d_residual_out=d["d_residual_out"])
    assert sorted(g) == ["dr", "dw"]
    for k in g:
        check(g[k], want[k], k)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_block_norm_in_place(types):
    import gated_delta_rule_69_amd as gdn
    c = _case(2, 13, 2568, types, seed=3)
    d = _device(c)
    args = lambda **over: {**{k: v for k, v in d.items() if k not in UPS}, **over}  # noqa: E731
    kw = dict(post_norm=True, activation="silu")
    r, n = gdn.gdn_block_norm_fwd(**args(), **kw)
    for target in ("y", "gate"):
        own = {k: d[k].clone() for k in ("residual", "y", "gate")}
        r2, n2 = gdn.gdn_block_norm_fwd(**args(**own), residual_out=own["residual"], out=own[target], **kw)
        assert r2 is own["residual"] and n2 is own[target]
        assert torch.equal(r2, r) and torch.equal(n2, n)


def test_block_norm_zero_huge_and_nan_rows():
    """A row of zeros gives zeros; magnitudes up to 1e18 in float32 do not overflow in the squares of
    what is normed; a NaN stays in its row."""
    import gated_delta_rule_69_amd as gdn
    from block_util import host
    from layer_util import check
    c = _case(1, 5, 1032, ("f32", "f32"), seed=4)
    c["residual"][0, 1] = 0
    c["y"][0, 1] = 0
    d, h = _device(c), host(c)
    ins = {k: v for k, v in d.items() if k not in UPS}
    r, n = gdn.gdn_block_norm_fwd(**ins, post_norm=True)
    want_r, want_n = block.block_norm(**{k: v for k, v in h.items() if k not in UPS}, post_norm=True)
    check(r, want_r, "r"), check(n, want_n, "n")
    assert (r[0, 1] == 0).all() and (n[0, 1] == 0).all()
    big, small = torch.full((1, 1, 64), 1e17, device=r.device), torch.full((1, 1, 64), 1e-15, device=r.device)
    for t in (big, small):
        _, n2 = gdn.gdn_block_norm_fwd(t, eps=0.0)
        assert (n2 - 1).abs().max() < 1e-6
    ins["y"] = d["y"].clone()
    ins["y"][0, 3, 70] = float("nan")
    r3, n3 = gdn.gdn_block_norm_fwd(**ins, post_norm=True)
    assert torch.isnan(r3[0, 3]).all() and torch.isnan(n3[0, 3]).all()
    keep = [0, 1, 2, 4]
    assert torch.equal(r3[:, keep], r[:, keep]) and torch.equal(n3[:, keep], n[:, keep])


def test_block_norm_streams_and_graph():
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    d = _device(_case(2, 700, 136, ("bf16", "f32"), seed=5))
    ins, ups = {k: v for k, v in d.items() if k not in UPS}, {k: d[k] for k in UPS}

    def work(**k):
        return list(gdn.gdn_block_norm_fwd(**ins, post_norm=True, **k)) + list(
            gdn.gdn_block_norm_bwd(**ins, **ups, post_norm=True, **k).values())

    want = work()
    torch.cuda.synchronize()
    both = [work(stream=torch.cuda.Stream(device=dev())) for _ in range(2)]
    torch.cuda.synchronize()
    for other in both + [work()]:
        for x, y in zip(want, other):
            assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for _ in range(4):
        d["y"].mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, work()):
            assert torch.equal(x, y)


def test_block_norm_of_no_tokens():
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    x, w = torch.zeros((2, 0, 64), device=dev()), torch.ones(64, device=dev())
    r, n = gdn.gdn_block_norm_fwd(x, x, x, weight=w)
    assert r.shape == n.shape == x.shape
    g = gdn.gdn_block_norm_bwd(x, x, x, weight=w, d_out=x)
    assert (g["dw"] == 0).all()


def test_block_norm_gradients_against_differences():
    """The kernels' own forward pass in float32: outputs are off by 2^-21 of their size, 2^-15 of it
    in a quotient over a step of 2^-7; checked to 1e-3 of the largest."""
    import gated_delta_rule_69_amd as gdn
    d = _device(_case(1, 3, 16, ("f32", "f32"), seed=6))
    ins, kw = {k: v for k, v in d.items() if k not in UPS}, dict(post_norm=True, activation="silu", residual_scale=0.6, eps=1e-2)

    def loss():
        r, n = gdn.gdn_block_norm_fwd(**ins, **kw)
        return ((r.double() * d["d_residual_out"].double()).sum() + (n.double() * d["d_out"].double()).sum()).item()

    g = gdn.gdn_block_norm_bwd(**ins, d_out=d["d_out"], d_residual_out=d["d_residual_out"], **kw)
    e = 2.0 ** -7
    for k, n in NAMES.items():
        flat, grad = d[n].view(-1), g[k].reshape(-1)
        for j in range(0, flat.numel(), max(1, flat.numel() // 9)):
            keep = flat[j].item()
            flat[j] = keep + e
            up = loss()
            flat[j] = keep - e
            down = loss()
            flat[j] = keep
            assert abs((up - down) / (2 * e) - grad[j].item()) < 1e-3 * grad.abs().max().item(), (n, j)


@pytest.mark.parametrize("C", [64, 2048, 16384])
def test_block_norm_up_to_the_largest_squares(C):
    """Values up to 1.8e19 / sqrt(C), whose squares add up to the largest float: norms of 1 before and after
    a block (a root, a reciprocal and two products of roundings: 1e-6), and finite gradients."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    big = torch.full((1, 2, C), 1.8e19 / C ** 0.5, device=dev())
    big[0, 1] = 1e-15
    for kw in (dict(), dict(y=big, post_norm=True)):
        _, n = gdn.gdn_block_norm_fwd(torch.zeros_like(big) if kw else big, eps=0.0, **kw)
        assert (n - 1).abs().max() < 1e-6
    g = gdn.gdn_block_norm_bwd(big, d_out=torch.ones_like(big), eps=0.0, weight=torch.ones(C, device=dev()))
    assert torch.isfinite(g["dr"]).all() and ((g["dw"] - 2).abs() < 1e-5).all()
