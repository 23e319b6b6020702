"""Block operators whose outputs take the place of an input: bit for bit what they give apart, or refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _conv_case(B, T, C, dt, seed=1):
    from layer_util import DTYPES, dev, rand
    gen = torch.Generator().manual_seed(seed)
    return (rand(gen, (B, T, C), DTYPES[dt]).to(dev()), rand(gen, (C, 4), torch.float32, 0.5).to(dev()),
            rand(gen, (B, 3, C), DTYPES[dt]).to(dev()))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,lens", [(1, 1, 8, None), (3, 2, 264, None), (5, 8, 520, [8, 0, 3, 1, 7]), (1030, 8, 8, None),
                                        (600, 5, 1024, None)])
def test_conv_of_few_tokens_in_place(B, T, C, lens, dt):
    import gated_delta_rule_69_amd as gdn
    from block_util import lengths
    x, w, s0 = _conv_case(B, T, C, dt)
    kw = dict(seq_lens=lengths(lens))
    y, end = gdn.gdn_short_conv_fwd(x, w, s0=s0, **kw)
    for step in (False, True):
        own, state = x.clone(), s0.clone()
        if step:
            got = gdn.gdn_short_conv_step(own, w, state=state, y=own, **kw)
        else:
            got, _ = gdn.gdn_short_conv_fwd(own, w, s0=state, s_final=state, y=own, **kw)
        assert got is own and torch.equal(state, end)
        for b in range(B if lens else 0):
            assert torch.equal(own[b, lens[b]:], x[b, lens[b]:])
            own[b, lens[b]:] = 0
        assert torch.equal(own, y)


def test_conv_of_more_tokens_is_refused_in_place():
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    x, w, s0 = _conv_case(2, 9, 16, "f32")
    keep = x.clone()
    for call in (lambda: gdn.gdn_short_conv_fwd(x, w, y=x), lambda: gdn.gdn_short_conv_step(x, w, state=s0, y=x)):
        with pytest.raises(gdn.GdnError):
            call()
    assert torch.equal(x, keep)
    # between the rows of a view there is room
    big = torch.zeros(8 * 512, device=dev())
    view, room = big.as_strided((1, 7, 64), (7 * 512, 512, 1)), big[64:512].view(1, 7, 64)
    x, w, _ = _conv_case(1, 7, 64, "f32")
    view.copy_(x)
    y, _ = gdn.gdn_short_conv_fwd(view, w, y=room)
    assert y is room and torch.equal(y, gdn.gdn_short_conv_fwd(x, w)[0]) and torch.equal(view, x)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["log", "sigmoid", "power"])
@pytest.mark.parametrize("B,T,C,lens", [(2, 1, 24, None), (2, 7, 40, [7, 3]), (1, 300, 24, None), (260, 300, 8, None),
                                        (2, 3000, 136, [3000, 1111])])
def test_scan_in_place(B, T, C, lens, gate, dt):
    """One token, tokens one by one, tiles, and segments side by side: h over x, f and i; gradients over x, f,
    i and d_h (through the C entry point, as the binding allocates them)."""
    import gated_delta_rule_69_amd as gdn
    from block_util import dev, lengths, scan_case
    from gated_delta_rule_69_amd import _block
    print(f"scan in place {B} {T} {C} {gate} {dt}", flush=True)
    c = {k: None if v is None else v.to(dev()) for k, v in scan_case(B, T, C, dt, gate, True, seed=T, lens=lens).items()}
    x, f, i, d_h = (c[n].nan_to_num() for n in ("x", "f", "i", "d_h"))
    kw = dict(gate=gate, decay=c["decay"], seq_lens=lengths(lens))
    live = torch.ones((B, T, 1), dtype=torch.bool, device=dev())
    for b, n in enumerate(lens or []):
        live[b, n:] = False
    want, end = gdn.gdn_gated_scan_fwd(x, f, i, h0=c["h0"], **kw)
    one = gdn.gdn_gated_scan_step(x, f, i, state=c["h0"].clone(), **kw)
    for k in range(3):
        own = [t.clone() for t in (x, f, i)]
        h, e = gdn.gdn_gated_scan_fwd(*own, h0=c["h0"], h=own[k], **kw)
        assert h is own[k] and torch.equal(torch.where(live, h, 0), want) and torch.equal(e, end)
        assert torch.equal(torch.where(live, 0, h), torch.where(live, 0, (x, f, i)[k]))
        own = [t.clone() for t in (x, f, i)]
        h = gdn.gdn_gated_scan_step(*own, state=c["h0"].clone(), h=own[k], **kw)
        assert torch.equal(torch.where(live, h, 0), one)
    grads = gdn.gdn_gated_scan_bwd(x, f, i, d_h=d_h, h0=c["h0"], dh_final=c["dh_final"], **kw)
    lib = _block._library()
    for turn in range(4):
        own = [t.clone() for t in (x, f, i, d_h)]
        to = [own[(turn + k) % 4] for k in range(3)]
        dd = None if c["decay"] is None else torch.empty_like(c["decay"])
        a = _block._scan_args(*own[:3], gate, c["decay"], kw["seq_lens"], c["h0"])
        ws = torch.empty(lib.gdn_gated_scan_bwd_workspace_bytes(a), dtype=torch.uint8, device=dev())
        g = _block._scan_grads_pack(*(t.data_ptr() for t in to), _block._at(dd), 0)
        assert lib.gdn_gated_scan_bwd(a, own[3].data_ptr(), c["dh_final"].data_ptr(), g, ws.data_ptr(), ws.numel(),
                                      torch.cuda.current_stream().cuda_stream) == 0
        for n, t in zip(("dx", "df", "di"), to):
            assert torch.equal(t, grads[n]), (turn, n)


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids="-".join)
@pytest.mark.parametrize("T,C", [(5, 64), (900, 2048), (300, 6144), (40, 12288)])
def test_block_norm_gradients_in_place(T, C, types):
    """dr over r or its upstream gradient, dy and dgate over y, gate and d_out (through the C entry point)."""
    import gated_delta_rule_69_amd as gdn
    from gated_delta_rule_69_amd import _block, _layer
    from layer_util import DTYPES, dev, rand
    print(f"norm in place {T} {C} {types}", flush=True)
    gen = torch.Generator().manual_seed(C)
    dt, rt = (DTYPES[t] for t in types)
    r, up_r = (rand(gen, (2, T, C), rt).to(dev()) for _ in range(2))
    y, gate, up = (rand(gen, (2, T, C), dt).to(dev()) for _ in range(3))
    w = rand(gen, (C,), torch.float32).to(dev())
    kw = dict(post_norm=True, weight=w, activation="silu")
    want = gdn.gdn_block_norm_bwd(r, y, gate, d_out=up, d_residual_out=up_r, **kw)
    lib = _block._library()
    for turn in range(3):
        rows, res = [t.clone() for t in (y, gate, up)], [t.clone() for t in (r, up_r)]
        dy, dgate, dr, dw = rows[turn], rows[(turn + 1) % 3], res[turn % 2], torch.empty_like(w)
        a = _block._norm_args(res[0], rows[0], rows[1], w, True, None, None, "silu", 1.0, 1e-6, dt)
        ws = torch.empty(lib.gdn_block_norm_bwd_workspace_bytes(a), dtype=torch.uint8, device=dev())
        g = _block._norm_grads_pack(res[1].data_ptr(), rows[2].data_ptr(), dr.data_ptr(), dy.data_ptr(), dgate.data_ptr(), 0, 0,
                                    dw.data_ptr())
        _layer._done(lib.gdn_block_norm_bwd(a, g, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream), "bwd")
        for n, t in (("dy", dy), ("dgate", dgate), ("dr", dr), ("dw", dw)):
            assert torch.equal(t, want[n]), (turn, n)
