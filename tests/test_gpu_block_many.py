"""Very many sequences and very wide rows through the tiled kernels of the block operators, forward and
gradients: grids of thousands of workgroups, sums over thousands of rows. The definition sees the sequences
side by side as channels of one."""
import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu


def _fold(t):
    """[B, T, C] -> [1, T, B C]."""
    return None if t is None else np.ascontiguousarray(t.transpose(1, 0, 2)).reshape(1, t.shape[1], -1)


def _unfold(t, B):
    return t.reshape(t.shape[1], B, -1).transpose(1, 0, 2)


@pytest.mark.parametrize("dt,B,T,C", [
    ("bf16", 4096, 129, 8), ("bf16", 3, 49, 16384), ("bf16", 1, 65, 65536), ("bf16", 4096, 300, 8),
    ("f32", 4096, 129, 8), ("f32", 3, 97, 16384), ("f32", 1, 129, 65536)])   # a token more than go one by one
@pytest.mark.parametrize("gate", ["log", "power"])
def test_scan_many(dt, B, T, C, gate):
    import gated_delta_rule_69_amd as gdn
    from block_util import dev, host, scan_case
    from layer_util import check
    print(f"many {dt} {B} {T} {C} {gate}", flush=True)
    c = scan_case(B, T, C, dt, gate, gate == "power", seed=B + T)
    d, h = {k: None if v is None else v.to(dev()) for k, v in c.items()}, host(c)
    kw = dict(gate=gate, decay=d["decay"], h0=d["h0"])
    out, end, marks = gdn.gdn_gated_scan_fwd(d["x"], d["f"], d["i"], want_checkpoints=True, **kw)
    x, f, i, up = (_fold(h[n]) for n in ("x", "f", "i", "d_h"))
    ref = dict(gate=gate, decay=None if h["decay"] is None else np.tile(h["decay"], B), h0=h["h0"].reshape(1, -1))
    want, want_end = block.scan_forward(x, f, i, **ref)
    check(out, _unfold(want, B), "h")
    check(end, want_end.reshape(B, C), "h_final")
    del want, out
    grads = block.scan_backward(x, f, i, d_h=up, dh_final=h["dh_final"].reshape(1, -1), **ref)
    for ck in (marks, None):
        g = gdn.gdn_gated_scan_bwd(d["x"], d["f"], d["i"], d_h=d["d_h"], dh_final=d["dh_final"], checkpoints=ck, **kw)
        for n, t in g.items():
            w = grads[n]
            check(t, w.reshape(B, C).sum(0) if n == "ddecay" else w.reshape(B, C) if n == "dh0" else _unfold(w, B), n)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C", [(4096, 3, 8), (4096, 40, 8), (1, 5, 65536), (2, 40, 65536), (1, 40000, 8)])
def test_conv_many(B, T, C, dt):
    import gated_delta_rule_69_amd as gdn
    from layer_util import DTYPES, check, dev, f64, rand
    print(f"conv many {dt} {B} {T} {C}", flush=True)
    gen, dtype = torch.Generator().manual_seed(T), DTYPES[dt]
    x, d_y, s0, ds = (rand(gen, (B, n, C), dtype) for n in (T, T, 3, 3))
    w, bias = rand(gen, (C, 4), torch.float32, 0.5), rand(gen, (C,), torch.float32, 0.3)
    X, Y, S, D, W, b = (t.to(dev()) for t in (x, d_y, s0, ds, w, bias))
    fold = dict(s0=_fold(f64(s0)), w=np.tile(f64(w), (B, 1)), bias=np.tile(f64(bias), B))
    y, end = gdn.gdn_short_conv_fwd(X, W, b, s0=S)
    want, want_end = block.conv_forward(_fold(f64(x)), **fold)
    check(y, _unfold(want, B), "y")
    check(end, _unfold(want_end, B), "s_final")
    ref = block.conv_backward(_fold(f64(x)), d_y=_fold(f64(d_y)), ds_final=_fold(f64(ds)), **fold)
    g = gdn.gdn_short_conv_bwd(X, W, b, d_y=Y, s0=S, ds_final=D)
    check(g["dx"], _unfold(ref["dx"], B), "dx")
    check(g["ds0"], _unfold(ref["ds0"], B), "ds0")
    check(g["dw"], ref["dw"].reshape(B, C, 4).sum(0), "dw")
    check(g["dbias"], ref["dbias"].reshape(B, C).sum(0), "dbias")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_as_far_apart_as_strides_go(dt):
    """Tokens 2^24 elements apart: a wave's last row starts 63 strides behind its first, 2^32 - 2^26 bytes in
    float32. Memory between the rows is not initialised: nothing may use it."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import DTYPES, check, dev, f64, rand
    T, C, ld = 200, 16, 1 << 24
    gen, dtype = torch.Generator().manual_seed(5), DTYPES[dt]
    x, d_h = (rand(gen, (1, T, C), dtype) for _ in range(2))
    f = (rand(gen, (1, T, C), torch.float32) + 2).to(dtype)
    big = torch.empty(T * ld, dtype=dtype, device=dev())
    X, F = (big.as_strided((1, T, C), (T * ld, ld, 1), o) for o in (0, ld - 64))
    X.copy_(x.to(dev())), F.copy_(f.to(dev()))
    want, want_end = block.scan_forward(f64(x), f64(f))
    h, end = gdn.gdn_gated_scan_fwd(X, F)
    check(h, want, "h")
    check(end, want_end, "end")
    ref, g = block.scan_backward(f64(x), f64(f), d_h=f64(d_h)), gdn.gdn_gated_scan_bwd(X, F, d_h=d_h.to(dev()))
    for n in ("dx", "df", "dh0"):
        check(g[n], ref[n], n)
    one = gdn.gdn_gated_scan_step(X, F, state=torch.zeros((1, C), device=dev()))
    check(one, want, "step")
    w = torch.ones((C, 3))
    check(gdn.gdn_short_conv_fwd(X, w.to(dev()), activation=None)[0], block.conv_forward(f64(x), f64(w), activation=None)[0], "conv")
    dx = gdn.gdn_short_conv_bwd(X, w.to(dev()), d_y=d_h.to(dev()), activation=None)
    back = block.conv_backward(f64(x), f64(w), d_y=f64(d_h), activation=None)
    check(dx["dx"], back["dx"], "conv dx")
    check(dx["dw"], back["dw"], "conv dw")
    r, n = gdn.gdn_block_norm_fwd(X, F)
    want_r, want_n = block.block_norm(f64(x), f64(f))
    check(r, want_r, "residual_out")
    check(n, want_n, "out")
    del big, X, F
