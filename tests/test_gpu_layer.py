"""The layer operators together, as a layer uses them: norms of queries and keys, linear
attention (or a delta rule), the gated norm, and the way back."""
import numpy as np
import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-5))


def _inputs(dt, B=2, T=150, H=4, Hk=2, dk=64, dv=64):
    """Projection output [B, T, q | k | v | gate], weights and tables, on the device."""
    from layer_util import DTYPES, dev, rand
    gen = torch.Generator().manual_seed(51)
    dtype = DTYPES[dt]
    sizes = [(Hk, dk), (Hk, dk), (H, dv), (H, dv)]
    x = rand(gen, (B, T, sum(h * d for h, d in sizes)), dtype).to(dev())
    q, k, v, gate = (p.unflatten(-1, s) for p, s in zip(torch.split(x, [h * d for h, d in sizes], -1), sizes))
    wq, wk, w = (1 + rand(gen, (d,), torch.float32, 0.2).to(dev()) for d in (dk, dk, dv))
    angle = torch.rand((T, dk // 4), generator=gen, dtype=torch.float64) * 6.3
    g = (-torch.exp2(torch.linspace(0, -7, H))).float().to(dev())
    return dict(q=q, k=k, v=v, gate=gate, wq=wq, wk=wk, w=w, cos=angle.cos().float().to(dev()),
                sin=angle.sin().float().to(dev()), g=g, dy=rand(gen, (B, T, H, dv), dtype).to(dev()))


def _norm_kw(t, norm="rms"):
    return dict(norm=norm, eps=1e-5, q_scale=0.125, cos=t["cos"], sin=t["sin"])


def _norm_ref(t, which, norm="rms", dy=None):
    from layer_util import f64
    return layer.head_norm(f64(t[which]), f64(t["w" + which]), norm=norm, eps=EPS, scale=0.125 if which == "q" else 1.0,
                           cos=f64(t["cos"]), sin=f64(t["sin"]), dy=dy)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_layer_forward_and_backward(dt):
    """Each stage against its definition on what the stage before it left."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, f64
    t = _inputs(dt)
    qn, kn = gdn.gdn_qk_norm_fwd(t["q"], t["k"], t["wq"], t["wk"], **_norm_kw(t))
    o, S = gdn.gdn_linear_chunk_fwd(qn, kn, t["v"], t["g"])
    y = gdn.gdn_gated_norm_fwd(o, t["gate"], t["w"], eps=1e-5)
    check(qn, _norm_ref(t, "q"), "q")
    check(kn, _norm_ref(t, "k"), "k")
    o_ref, S_ref = layer.linear_forward(f64(qn), f64(kn), f64(t["v"]), f64(t["g"]))
    check(o, o_ref, "o")
    check(S, S_ref, "state")
    y_ref, do_ref, dgate_ref, dw_ref = layer.gated_norm(f64(o), f64(t["gate"]), f64(t["w"]), eps=EPS, dy=f64(t["dy"]))
    check(y, y_ref, "y")

    out = gdn.gdn_gated_norm_bwd(o, t["gate"], t["w"], d_out=t["dy"], eps=1e-5)
    check(out["dx"], do_ref, "do")
    check(out["dgate"], dgate_ref, "dgate")
    check(out["dw"], dw_ref, "dw")
    lin = gdn.gdn_linear_chunk_bwd(qn, kn, t["v"], t["g"], d_o=out["dx"])
    ref = layer.linear_backward(f64(qn), f64(kn), f64(t["v"]), f64(t["g"]), f64(out["dx"]))
    for name in ("dq", "dk", "dv", "ds0"):
        check(lin[name], ref[name], name)
    back = gdn.gdn_qk_norm_bwd(t["q"], t["k"], t["wq"], t["wk"], dq_out=lin["dq"], dk_out=lin["dk"], **_norm_kw(t))
    for which in ("q", "k"):
        _, dx, dw = _norm_ref(t, which, dy=f64(lin["d" + which]))
        check(back["d" + which], dx, "d" + which)
        check(back["dw" + which], dw, "dw" + which)

    # a prompt and then single tokens: the states and rows of one longer prompt
    if dt == "f32":
        cut = 147
        o1, state = gdn.gdn_linear_chunk_fwd(*(x[:, :cut].contiguous() for x in (qn, kn, t["v"])), t["g"])
        rows = [gdn.gdn_linear_recurrent_step(*(x[:, i:i + 1].contiguous() for x in (qn, kn, t["v"])), t["g"], state=state)
                for i in range(cut, 150)]
        check(torch.cat([o1, *rows], 1), o_ref, "o in parts")
        check(state, S_ref, "state in parts")


def test_delta_rule_layer_with_unit_keys():
    """The GDN delta rule between L2 norms of its queries and keys and the gated norm, with
    its float32 gradients taken back through the norms."""
    import gated_delta_rule_69_amd as gdn
    import oracle
    from layer_util import check, f64
    t = _inputs("bf16", Hk=4)
    B, T, H, d = t["v"].shape
    gen = torch.Generator().manual_seed(52)
    alpha = torch.sigmoid(3 + torch.randn((B, T, H), generator=gen)).to(t["v"])
    beta = torch.sigmoid(torch.randn((B, T, H), generator=gen)).to(t["v"])
    v = t["v"].contiguous()
    qn, kn = gdn.gdn_qk_norm_fwd(t["q"], t["k"], norm="l2", eps=1e-5, q_scale=0.125)
    for name, x in (("q", qn), ("k", kn)):
        check(x, layer.head_norm(f64(t[name]), norm="l2", eps=EPS, scale=0.125 if name == "q" else 1.0), name)
    o, _ = gdn.gdn_chunk_fwd("gdn", qn, kn, v, alpha, beta)
    inp = dict(variant="gdn", B=B, T=T, H=H, dk=d, dv=d, n_h=1, dtype="bf16", q=f64(qn), k=f64(kn), v=f64(v),
               alpha=f64(alpha), beta=f64(beta))
    o_ref, _ = oracle.forward(inp)
    assert oracle.rel_l2(f64(o), o_ref) <= 5e-3
    y = gdn.gdn_gated_norm_fwd(o, t["gate"], t["w"], eps=1e-5, activation="sigmoid")
    y_ref, do_ref, _, _ = layer.gated_norm(f64(o), f64(t["gate"]), f64(t["w"]), eps=EPS, activation="sigmoid", dy=f64(t["dy"]))
    check(y, y_ref, "y")
    back = gdn.gdn_gated_norm_bwd(o, t["gate"], t["w"], d_out=t["dy"], eps=1e-5, activation="sigmoid")
    check(back["dx"], do_ref, "do")
    g = gdn.gdn_recurrent_bwd("gdn", qn, kn, v, alpha, beta, d_o=back["dx"])
    assert g["dq"].dtype == torch.float32
    through = gdn.gdn_qk_norm_bwd(t["q"], t["k"], dq_out=g["dq"], dk_out=g["dk"], norm="l2", eps=1e-5, q_scale=0.125)
    for name in ("q", "k"):
        _, dx, _ = layer.head_norm(f64(t[name]), norm="l2", eps=EPS, scale=0.125 if name == "q" else 1.0, dy=f64(g["d" + name]))
        check(through["d" + name], dx, "d" + name)


def test_whole_layer_against_automatic_gradients():
    """float32, end to end: the chain's outputs and gradients against float64 autograd of the
    layer's formulas. Three stages of 1e-5 each, and a factor of 2 for their interplay."""
    import gated_delta_rule_69_amd as gdn
    import oracle
    from layer_util import f64
    t = _inputs("f32", T=70)
    qn, kn = gdn.gdn_qk_norm_fwd(t["q"], t["k"], t["wq"], t["wk"], **_norm_kw(t))
    o, _ = gdn.gdn_linear_chunk_fwd(qn, kn, t["v"], t["g"])
    y = gdn.gdn_gated_norm_fwd(o, t["gate"], t["w"], eps=1e-5)
    gate = gdn.gdn_gated_norm_bwd(o, t["gate"], t["w"], d_out=t["dy"], eps=1e-5)
    lin = gdn.gdn_linear_chunk_bwd(qn, kn, t["v"], t["g"], d_o=gate["dx"])
    back = gdn.gdn_qk_norm_bwd(t["q"], t["k"], t["wq"], t["wk"], dq_out=lin["dq"], dk_out=lin["dk"], **_norm_kw(t))
    got = dict(q=back["dq"], k=back["dk"], v=lin["dv"], gate=gate["dgate"], wq=back["dwq"], wk=back["dwk"], w=gate["dw"])

    leaf = {n: t[n].double().cpu().requires_grad_() for n in got}
    cos, sin = (t[n].double().cpu()[None, :, None] for n in ("cos", "sin"))

    def normed(x, w, scale):
        n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        r = cos.shape[-1]
        a, b = n[..., :r], n[..., r:2 * r]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, n[..., 2 * r:]), -1) * scale
    q, k = normed(leaf["q"], leaf["wq"], 0.125), normed(leaf["k"], leaf["wk"], 1.0)
    q, k = q.repeat_interleave(2, 2), k.repeat_interleave(2, 2)
    T = q.shape[1]
    i = torch.arange(T)
    decay = torch.exp(t["g"].double().cpu()[:, None, None] * (i[:, None] - i).clamp(min=0)) * (i[:, None] >= i)
    scores = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1).contiguous()) * decay
    of = torch.matmul(scores, leaf["v"].transpose(1, 2)).transpose(1, 2)
    ref = of * torch.rsqrt((of * of).mean(-1, keepdim=True) + EPS) * leaf["w"] * torch.nn.functional.silu(leaf["gate"])
    assert oracle.rel_l2(f64(y), ref.detach().numpy()) <= 6e-5
    ref.backward(t["dy"].double().cpu())
    for name in got:
        e = oracle.rel_l2(f64(got[name]), leaf[name].grad.numpy())
        assert e <= 6e-5, (name, e)


def test_padded_batch_through_the_layer():
    """A padded batch, outputs allocated by the calls, from memory that holds NaN: what lies
    behind the lengths reaches neither the rows nor a gradient of what lies before them."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, dev, f64
    t = _inputs("f32")
    B, T = t["v"].shape[:2]
    lens = [T, 43]
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev())
    shape, dy = t["v"].shape, t["dy"].clone()
    dy[1, lens[1]:] = 0
    q, k, v, gate = (t[n].contiguous() for n in ("q", "k", "v", "gate"))

    def leave_nan():  # the allocator hands this block out again
        torch.cuda.synchronize()
        torch.full(shape, float("nan"), device=dev())

    state = torch.zeros((B, shape[2], q.shape[3], shape[3]), device=dev())
    leave_nan()
    o, _ = gdn.gdn_linear_chunk_fwd(q, k, v, t["g"], seq_lens=seq_lens)
    leave_nan()
    o2 = gdn.gdn_linear_recurrent_step(q, k, v, t["g"], state=state, seq_lens=seq_lens)
    want, _ = layer.linear_forward(f64(q), f64(k), f64(v), f64(t["g"]), lens=lens)
    for x in (o, o2):
        assert (x[1, lens[1]:] == 0).all()
        check(x, want, "o")
    y = gdn.gdn_gated_norm_fwd(o, gate, t["w"], eps=1e-5)
    back = gdn.gdn_gated_norm_bwd(o, gate, t["w"], d_out=dy, eps=1e-5)
    ref = layer.gated_norm(f64(o), f64(gate), f64(t["w"]), eps=EPS, dy=f64(dy))
    for got, r, name in zip((y, back["dx"], back["dgate"], back["dw"]), ref, ("y", "do", "dgate", "dw")):
        check(got, r, name)


def test_results_do_not_depend_on_what_runs_beside_them():
    """Two calls at once on two streams, and twice the same call: equal bits."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    t = _inputs("bf16")
    qn, kn = gdn.gdn_qk_norm_fwd(t["q"], t["k"], t["wq"], t["wk"], **_norm_kw(t))
    kw = dict(dq_out=torch.randn_like(qn), dk_out=torch.randn_like(kn), **_norm_kw(t))
    run = lambda s: (gdn.gdn_linear_chunk_fwd(qn, kn, t["v"], t["g"], stream=s),  # noqa: E731
                     gdn.gdn_linear_chunk_bwd(qn, kn, t["v"], t["g"], d_o=t["dy"], stream=s),
                     gdn.gdn_qk_norm_bwd(t["q"], t["k"], t["wq"], t["wk"], stream=s, **kw),
                     gdn.gdn_gated_norm_bwd(t["v"], t["gate"], t["w"], d_out=t["dy"], stream=s))
    want = run(None)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(device=dev()) for _ in range(2)]
    both = [run(s) for s in sides]
    for s in sides:
        s.synchronize()
    for got in both:
        for w, g in zip(want, got):
            pairs = zip(w.values(), g.values()) if isinstance(w, dict) else zip(w, g)
            assert all(torch.equal(a, b) for a, b in pairs)


def test_norms_in_a_captured_graph():
    import gated_delta_rule_69_amd as gdn
    t = _inputs("bf16")
    kw = _norm_kw(t)
    dq, dk = torch.randn_like(t["q"].contiguous()), torch.randn_like(t["k"].contiguous())
    calls = lambda: (gdn.gdn_qk_norm_fwd(t["q"], t["k"], t["wq"], t["wk"], **kw)  # noqa: E731
                     + tuple(gdn.gdn_qk_norm_bwd(t["q"], t["k"], t["wq"], t["wk"], dq_out=dq, dk_out=dk, **kw).values())
                     + (gdn.gdn_gated_norm_fwd(t["v"], t["gate"], t["w"]),)
                     + tuple(gdn.gdn_gated_norm_bwd(t["v"], t["gate"], t["w"], d_out=t["dy"]).values()))
    want = calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        again = calls()
        for w, g, a in zip(want, got, again):
            assert torch.equal(w, g) and torch.equal(w, a)


def test_binding_refuses_tensors_that_do_not_fit():
    """Other types, shapes, strides and devices are refused before anything is launched."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    from gated_delta_rule_69_amd import GdnError
    x = torch.zeros((2, 10, 4, 32), device=dev())
    k, g, state = x[:, :, :2].contiguous(), torch.zeros(4, device=dev()), torch.zeros((2, 4, 32, 32), device=dev())
    lens, w, half = torch.ones(2, dtype=torch.int32, device=dev()), torch.ones(32, device=dev()), x.half()
    off = torch.zeros(x.numel() + 1, device=dev())[1:].view(x.shape)   # 4 bytes off a 16-byte border
    table = torch.zeros((10, 16), device=dev())
    linear = [("q", x), ("q", k.bfloat16()), ("k", k[:, :5]), ("k", k[0]), ("k", k.cpu()), ("v", half), ("v", x[0]),
              ("v", off), ("v", x.transpose(1, 2)), ("log_decay", g[:2]), ("log_decay", g.double()),
              ("log_decay", g.cpu()), ("seq_lens", lens.long()), ("seq_lens", lens[:1])]
    chunk = [("o", x.bfloat16()), ("o", k), ("o", x.transpose(2, 3)), ("o", off), ("s0", state[:1]),
             ("s0", state.bfloat16()), ("s_final", state.transpose(2, 3)), ("s_final", state.cpu()),
             ("workspace", torch.empty(16, dtype=torch.uint8, device=dev()))]
    step = [("o", k), ("o", x.cpu()), ("state", state[:1]), ("state", state.bfloat16())]
    back = [("d_o", x.bfloat16()), ("d_o", k), ("ds_final", state[:1]), ("s0", state.double())]
    norm = [("q", half), ("k", k[:1]), ("wq", w[:16]), ("wk", w.bfloat16()), ("cos", table[:9]), ("cos", None),
            ("sin", table[:, :8]), ("positions", torch.zeros((2, 10), dtype=torch.int64, device=dev())),
            ("norm", "max"), ("eps", -1.0), ("q_out", k), ("k_out", k.bfloat16()), ("q", off)]
    gate = [("x", half), ("gate", k), ("gate", x.bfloat16()), ("weight", w[:8]), ("activation", "tanh"), ("out", k),
            ("eps", float("nan")), ("gate", off)]
    base = dict(q=k, k=k, v=x, log_decay=g, seq_lens=lens)
    rope = dict(q=x, k=k, wq=w, wk=w, cos=table, sin=table)
    gated = dict(x=x, gate=x, weight=w)
    for fn, args, bad in ((gdn.gdn_linear_chunk_fwd, base, linear + chunk),
                          (gdn.gdn_linear_recurrent_step, dict(base, state=state), linear + step),
                          (gdn.gdn_linear_chunk_bwd, dict(base, d_o=x), linear + back),
                          (gdn.gdn_qk_norm_fwd, rope, norm),
                          (gdn.gdn_qk_norm_bwd, dict(rope, dq_out=x, dk_out=k),
                           norm[:-4] + [("dq_out", k), ("dk_out", k.bfloat16())]),
                          (gdn.gdn_gated_norm_fwd, gated, gate),
                          (gdn.gdn_gated_norm_bwd, dict(gated, d_out=x), gate[:5] + [("d_out", k), ("d_out", half)])):
        fn(**args)  # as they are they fit
        for name, value in bad:
            with pytest.raises((ValueError, GdnError)):
                fn(**{**args, name: value})
                print(fn.__name__, name, "was taken", flush=True)
