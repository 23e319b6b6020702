"""The block operators together, as a model's layers call them: norm, projection, convolution,
gated recurrence (or the delta rule), gate, norm with the residual; prompts, single tokens and
gradients against float64."""
import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu

B, T, C, W = 2, 150, 64, 4


def _weights(gen):
    from layer_util import rand
    f32 = torch.float32
    one = lambda s=0.1: (1 + rand(gen, (C,), f32, s)).float()  # noqa: E731
    return dict(w_in=one(), proj=rand(gen, (C, 4 * C), f32, C ** -0.5), conv=rand(gen, (C, W), f32, 0.5), bias=rand(gen, (C,), f32, 0.1),
                decay=torch.exp(2 * torch.rand(C, generator=gen) - 3), w_post=one(), scale=one(), w_next=one())


def _layer(gdn, p, x, carry=None):
    """One layer on x [B, T, C] float32; ``carry`` (convolution's state, recurrence's state) is
    updated for decoding. Returns the residual, the next input and what the gradients need."""
    _, n = gdn.gdn_block_norm_fwd(x, weight=p["w_in"])
    z = n @ p["proj"]
    v, f, i, gate = z.split(C, -1)
    if carry is None:
        c, _ = gdn.gdn_short_conv_fwd(v, p["conv"], p["bias"])
        h, _, marks = gdn.gdn_gated_scan_fwd(c, f, i, gate="power", decay=p["decay"], want_checkpoints=True)
    else:
        c = gdn.gdn_short_conv_step(v, p["conv"], p["bias"], state=carry[0])
        h, marks = gdn.gdn_gated_scan_step(c, f, i, state=carry[1], gate="power", decay=p["decay"]), None
    r, out = gdn.gdn_block_norm_fwd(x, h, gate, weight=p["w_next"], post_norm=True, post_weight=p["w_post"], scale=p["scale"],
                                    activation="silu")
    return r, out, (n, v, f, i, gate, c, h, marks)


def _oracle(p, x):
    f = {k: v.double().cpu().numpy() for k, v in p.items()}
    x = x.double().cpu().numpy()
    _, n = block.block_norm(x, weight=f["w_in"])
    v, g, i, gate = np.split(n @ f["proj"], 4, -1)
    c, _ = block.conv_forward(v, f["conv"], f["bias"])
    h, _ = block.scan_forward(c, g, i, gate="power", decay=f["decay"])
    r, out = block.block_norm(x, h, gate, weight=f["w_next"], post_norm=True, post_weight=f["w_post"], scale=f["scale"], activation="silu")
    return f, x, n, v, g, i, gate, c, h, r, out


def test_layer_prompt_and_decoding():
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, dev
    gen = torch.Generator().manual_seed(1)
    p = {k: v.to(dev()) for k, v in _weights(gen).items()}
    x = torch.randn((B, T, C), generator=gen).to(dev())
    *_, want_r, want_out = _oracle(p, x)
    r, out, _ = _layer(gdn, p, x)
    check(r, want_r, "residual")
    check(out, want_out, "next input")
    # a prompt of 120 tokens, then token by token from its states
    head = x[:, :120].contiguous()
    _, n = gdn.gdn_block_norm_fwd(head, weight=p["w_in"])
    v, f, i, _ = (n @ p["proj"]).split(C, -1)
    c, s_conv = gdn.gdn_short_conv_fwd(v, p["conv"], p["bias"])
    _, s_scan = gdn.gdn_gated_scan_fwd(c, f, i, gate="power", decay=p["decay"])
    rows = []
    for t in range(120, T):
        _, one, _ = _layer(gdn, p, x[:, t:t + 1].contiguous(), carry=(s_conv, s_scan))
        rows.append(one)
    check(torch.cat(rows, 1), want_out[:, 120:], "decoded")


def test_layer_gradients():
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, dev
    gen = torch.Generator().manual_seed(2)
    p = {k: v.to(dev()) for k, v in _weights(gen).items()}
    x, d_r, d_out = (torch.randn((B, T, C), generator=gen).to(dev()) for _ in range(3))
    _, _, (n, v, f, i, gate, c, h, marks) = _layer(gdn, p, x)
    g = gdn.gdn_block_norm_bwd(x, h, gate, d_out=d_out, d_residual_out=d_r, weight=p["w_next"], post_norm=True,
                               post_weight=p["w_post"], scale=p["scale"], activation="silu")
    s = gdn.gdn_gated_scan_bwd(c, f, i, d_h=g["dy"], gate="power", decay=p["decay"], checkpoints=marks)
    k = gdn.gdn_short_conv_bwd(v, p["conv"], p["bias"], d_y=s["dx"])
    dz = torch.cat((k["dx"], s["df"], s["di"], g["dgate"]), -1)
    first = gdn.gdn_block_norm_bwd(x, weight=p["w_in"], d_out=dz @ p["proj"].T, d_residual_out=g["dr"])
    w, xd, nd, vd, fd, idd, gd, cd, hd, _, _ = _oracle(p, x)
    ur, uo = d_r.double().cpu().numpy(), d_out.double().cpu().numpy()
    G = block.block_norm(xd, hd, gd, weight=w["w_next"], post_norm=True, post_weight=w["w_post"], scale=w["scale"], activation="silu",
                         d_residual_out=ur, d_out=uo)[2]
    S = block.scan_backward(cd, fd, idd, d_h=G["dy"], gate="power", decay=w["decay"])
    K = block.conv_backward(vd, w["conv"], w["bias"], d_y=S["dx"])
    DZ = np.concatenate((K["dx"], S["df"], S["di"], G["dgate"]), -1)
    F = block.block_norm(xd, weight=w["w_in"], d_out=DZ @ w["proj"].T, d_residual_out=G["dr"])[2]
    for name, got, want in (("dx", first["dr"], F["dr"]), ("dw_in", first["dw"], F["dw"]), ("dz", dz, DZ), ("dconv", k["dw"], K["dw"]),
                            ("dbias", k["dbias"], K["dbias"]), ("ddecay", s["ddecay"], S["ddecay"]), ("dscale", g["dscale"], G["dscale"]),
                            ("dw_post", g["dw_post"], G["dw_post"]), ("dw_next", g["dw"], G["dw"])):
        check(got, want, name)


def test_convolution_before_the_delta_rule():
    """q, k and v through one convolution, normed, into the chunked delta rule: the views go from one
    operator into the next, and the padded batch's rows behind the lengths stay out of every sum."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import check, dev, f64
    H, d = 2, 32
    gen = torch.Generator().manual_seed(3)
    lens = [T, 61]
    x = torch.randn((B, T, 3 * H * d), generator=gen)
    x[1, 61:] = float("nan")
    w, log_decay = torch.randn((3 * H * d, W), generator=gen) * 0.5, -torch.rand(H, generator=gen)
    L = torch.tensor(lens, dtype=torch.int32, device=dev())
    y, _ = gdn.gdn_short_conv_fwd(x.to(dev()), w.to(dev()), seq_lens=L)
    q, k, v = (t.unflatten(-1, (H, d)) for t in y.split(H * d, -1))
    q, k = gdn.gdn_qk_norm_fwd(q, k, norm="l2", eps=1e-6)
    o, end = gdn.gdn_linear_chunk_fwd(q, k, v, log_decay.to(dev()), seq_lens=L)
    from oracle import layer
    Y, _ = block.conv_forward(f64(x), f64(w), lens=lens)
    Q, K, V = (t.reshape(B, T, H, d) for t in np.split(Y, 3, -1))
    Q, K = (layer.head_norm(t, norm="l2", eps=1e-6) for t in (Q, K))
    want, want_end = layer.linear_forward(Q, K, V, f64(log_decay), lens=lens)
    check(o, want, "o")
    check(end, want_end, "state")
