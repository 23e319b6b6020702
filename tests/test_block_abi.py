"""Host-side argument checks of the block operators: the documented status, before any launch
(no GPU is touched), and the binding's own refusals."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # an aligned, never-dereferenced address
BIG = 1 << 44


@pytest.fixture(scope="module")
def lib():
    import os
    from gated_delta_rule_69_amd import _block, _lib
    if not os.path.exists(_lib.LIB_PATH):
        from gated_delta_rule_69_amd import build
        build.build()
    return _block._library()


def _of(structure, over, **fields):
    return ctypes.byref(structure(**{**fields, **over}))


def scan(**over):
    from gated_delta_rule_69_amd._block import GdnScanArgs
    return _of(GdnScanArgs, over, dtype=1, gate=2, B=2, T=100, C=64, x=FAKE, f=FAKE, h=2 * FAKE)


def conv(**over):
    from gated_delta_rule_69_amd._block import GdnConvArgs
    return _of(GdnConvArgs, over, dtype=1, activation=1, B=2, T=100, C=64, W=4, x=FAKE, w=FAKE, y=2 * FAKE)


def norm(**over):
    from gated_delta_rule_69_amd._block import GdnBlockNormArgs
    return _of(GdnBlockNormArgs, over, dtype=1, residual_dtype=1, activation=2, post_norm=1, B=2, T=100, C=64, eps=1e-6,
               residual_scale=1.0, r=FAKE, y=2 * FAKE, gate=3 * FAKE, scale=FAKE, post_weight=FAKE, weight=FAKE,
               residual_out=4 * FAKE, out=5 * FAKE)


SIZES = [("dtype", 2, -1), ("B", 0, -1), ("T", -1, -1), ("C", 0, -1), ("C", 12, -1), ("C", -8, -1), ("B", 1 << 21, -2),
         ("C", (1 << 16) + 8, -2), ("T", 1 << 31, -2), ("B", 1 << 19, -2), ("x_stride", 56, -1), ("x_stride", 68, -1),
         ("x_stride", -64, -1), ("x_stride", 1 << 25, -2)]


@pytest.mark.parametrize("field,value,status", SIZES + [
    ("gate", 0, -1), ("gate", 4, -1), ("f_stride", 8, -1), ("i_stride", 70, -1), ("x", 0, -1), ("x", FAKE + 8, -1), ("f", 0, -1),
    ("f", FAKE + 4, -1), ("i", FAKE + 8, -1), ("decay", FAKE, -1), ("gate", 3, -1), ("seq_lens", FAKE + 2, -1), ("h", 0, -1),
    ("h", FAKE + 8, -1)])
def test_scan_refusals(lib, field, value, status):
    a = scan(**{field: value})
    assert lib.gdn_gated_scan_fwd(a, FAKE, BIG, None) == status
    assert lib.gdn_gated_scan_step(a, FAKE, None) == status
    if (field, value, status) in SIZES:
        assert lib.gdn_gated_scan_workspace_bytes(a) == 0 and lib.gdn_gated_scan_bwd_workspace_bytes(a) == 0


def test_scan_workspace_and_state_checks(lib):
    need = lib.gdn_gated_scan_workspace_bytes(scan())
    assert need > 0
    assert lib.gdn_gated_scan_fwd(scan(), None, 0, None) == -3
    assert lib.gdn_gated_scan_fwd(scan(), FAKE, need - 1, None) == -3
    assert lib.gdn_gated_scan_fwd(scan(), FAKE + 16, need, None) == -3
    for field in ("h0", "h_final", "checkpoints"):
        assert lib.gdn_gated_scan_fwd(scan(**{field: FAKE + 8}), FAKE, BIG, None) == -1
    assert lib.gdn_gated_scan_fwd(None, FAKE, BIG, None) == -1
    assert lib.gdn_gated_scan_step(scan(), None, None) == -1 and lib.gdn_gated_scan_step(scan(), FAKE + 4, None) == -1
    none = dict(T=0, x=0, f=0, h=0)
    assert lib.gdn_gated_scan_fwd(scan(**none), FAKE, BIG, None) == 0
    assert lib.gdn_gated_scan_step(scan(**none), FAKE, None) == 0


def test_scan_backward_checks(lib):
    from gated_delta_rule_69_amd._block import GdnScanGrads
    full = dict(dx=FAKE, df=FAKE, di=0, ddecay=0, dh0=FAKE)
    need = lib.gdn_gated_scan_bwd_workspace_bytes(scan())
    assert need > lib.gdn_gated_scan_workspace_bytes(scan())
    call = lambda a=None, n=BIG, ws=FAKE, dh=FAKE, end=None, **over: lib.gdn_gated_scan_bwd(  # noqa: E731
        a or scan(), dh, end, ctypes.byref(GdnScanGrads(**{**full, **over})), ws, n, None)
    assert call(n=need - 1) == -3 and call(ws=None) == -3 and call(ws=FAKE + 16) == -3
    assert call(dh=None) == -1 and call(dh=FAKE + 2) == -1 and call(end=FAKE + 8) == -1
    for field in ("dx", "df"):
        assert call(**{field: 0}) == -1 and call(**{field: FAKE + 4}) == -1
    assert call(dh0=FAKE + 4) == -1 and call(a=scan(h0=FAKE + 4)) == -1 and call(a=scan(checkpoints=FAKE + 8)) == -1
    assert call(di=FAKE) == -1                                   # no i
    assert call(a=scan(i=FAKE)) == -1                            # i, and nowhere for its gradient
    assert call(ddecay=FAKE) == -1                               # not the power gate
    assert call(a=scan(gate=3, decay=FAKE), ddecay=FAKE + 8) == -1
    assert lib.gdn_gated_scan_bwd(scan(), FAKE, None, None, FAKE, BIG, None) == -1
    assert call(a=scan(T=0, x=0, f=0), dh=None, dx=0, df=0, dh0=0) == 0


@pytest.mark.parametrize("field,value,status", SIZES + [
    ("activation", 2, -1), ("activation", 3, -1), ("W", 1, -2), ("W", 5, -2), ("x", 0, -1), ("x", FAKE + 8, -1), ("w", 0, -1),
    ("w", FAKE + 8, -1), ("bias", FAKE + 4, -1), ("seq_lens", FAKE + 1, -1), ("y", 0, -1), ("y", FAKE + 4, -1)])
def test_conv_refusals(lib, field, value, status):
    a = conv(**{field: value})
    assert lib.gdn_short_conv_fwd(a, None) == status
    assert lib.gdn_short_conv_step(a, FAKE, None) == status


def test_conv_state_and_backward_checks(lib):
    from gated_delta_rule_69_amd._block import GdnConvGrads
    assert lib.gdn_short_conv_fwd(conv(s0=FAKE + 8), None) == -1 and lib.gdn_short_conv_fwd(conv(s_final=FAKE + 8), None) == -1
    assert lib.gdn_short_conv_step(conv(), None, None) == -1 and lib.gdn_short_conv_step(conv(), FAKE + 8, None) == -1
    assert lib.gdn_short_conv_fwd(None, None) == -1
    assert lib.gdn_short_conv_fwd(conv(T=0, x=0, y=0), None) == 0 and lib.gdn_short_conv_step(conv(T=0, x=0, y=0), FAKE, None) == 0
    full = dict(dx=FAKE, dw=FAKE, dbias=0, ds0=FAKE)
    need = lib.gdn_short_conv_bwd_workspace_bytes(conv())
    call = lambda a=None, n=BIG, ws=FAKE, dy=FAKE, end=None, **over: lib.gdn_short_conv_bwd(  # noqa: E731
        a or conv(), dy, end, ctypes.byref(GdnConvGrads(**{**full, **over})), ws, n, None)
    assert need > 0 and lib.gdn_short_conv_bwd_workspace_bytes(conv(W=5)) == 0
    assert call(n=need - 1) == -3 and call(ws=None) == -3 and call(ws=FAKE + 8) == -3
    assert call(dy=None) == -1 and call(dy=FAKE + 8) == -1 and call(end=FAKE + 8) == -1 and call(dx=0) == -1
    assert call(dw=FAKE + 2) == -1 and call(ds0=FAKE + 8) == -1 and call(dbias=FAKE) == -1 and call(a=conv(w=0)) == -1
    assert lib.gdn_short_conv_bwd(conv(), FAKE, None, None, FAKE, BIG, None) == -1
    assert call(a=conv(T=0, x=0), dy=None, dx=0, dw=0, ds0=0) == 0


@pytest.mark.parametrize("field,value,status", [s for s in SIZES if s[0] != "x_stride"] + [
    ("C", 16392, -2), ("residual_dtype", 2, -1), ("activation", 0, -1), ("post_norm", 2, -1), ("eps", -1.0, -1),
    ("eps", float("nan"), -1), ("residual_scale", float("inf"), -1), ("r_stride", 56, -1), ("y_stride", 68, -1),
    ("gate_stride", 1 << 25, -2), ("r", 0, -1), ("r", FAKE + 8, -1), ("y", 0, -1), ("gate", FAKE + 8, -1),
    ("scale", FAKE + 4, -1), ("post_weight", FAKE + 8, -1), ("post_norm", 0, -1), ("weight", FAKE + 8, -1),
    ("out", FAKE + 8, -1), ("residual_out", FAKE + 8, -1), ("out", 4 * FAKE, -1)])
def test_block_norm_refusals(lib, field, value, status):
    a = norm(**{field: value})
    assert lib.gdn_block_norm_fwd(a, None) == status
    if status == -2 or field in ("C", "dtype", "B", "T", "residual_dtype", "activation", "eps", "residual_scale"):
        assert lib.gdn_block_norm_bwd_workspace_bytes(a) == 0


def test_block_norm_in_place_and_missing_inputs(lib):
    assert lib.gdn_block_norm_fwd(norm(out=0, residual_out=0), None) == -1
    assert lib.gdn_block_norm_fwd(norm(r_stride=128, residual_out=FAKE), None) == -1
    assert lib.gdn_block_norm_fwd(norm(y_stride=128, out=2 * FAKE), None) == -1
    assert lib.gdn_block_norm_fwd(norm(gate_stride=128, out=3 * FAKE), None) == -1
    assert lib.gdn_block_norm_fwd(norm(residual_dtype=0, out=FAKE), None) == -1          # another type's rows
    assert lib.gdn_block_norm_fwd(norm(residual_dtype=0, residual_out=2 * FAKE), None) == -1
    for over in (dict(gate=FAKE), dict(scale=FAKE), dict(post_norm=1), dict(post_weight=FAKE)):
        assert lib.gdn_block_norm_fwd(norm(**{**dict(y=0, gate=0, scale=0, post_norm=0, post_weight=0), **over}), None) == -1
    assert lib.gdn_block_norm_fwd(norm(T=0, r=0, y=0, gate=0, out=0, residual_out=0), None) == 0
    assert lib.gdn_block_norm_fwd(None, None) == -1


def test_block_norm_backward_checks(lib):
    from gated_delta_rule_69_amd._block import GdnBlockNormGrads
    full = dict(d_residual_out=FAKE, d_out=FAKE, dr=FAKE, dy=FAKE, dgate=FAKE, dscale=FAKE, dpost_weight=FAKE, dweight=FAKE)
    need = lib.gdn_block_norm_bwd_workspace_bytes(norm())
    call = lambda a=None, n=BIG, ws=FAKE, **over: lib.gdn_block_norm_bwd(  # noqa: E731
        a or norm(), ctypes.byref(GdnBlockNormGrads(**{**full, **over})), ws, n, None)
    assert need > 0
    assert call(n=need - 1) == -3 and call(ws=None) == -3 and call(ws=FAKE + 8) == -3
    assert call(d_residual_out=0, d_out=0) == -1
    for field in ("d_residual_out", "d_out", "dr", "dy", "dgate"):
        assert call(**{field: FAKE + 8}) == -1
    for field in ("dscale", "dpost_weight", "dweight"):
        assert call(**{field: FAKE + 2}) == -1
    bare = dict(y=0, gate=0, scale=0, post_norm=0, post_weight=0)
    left = dict(dy=0, dgate=0, dscale=0, dpost_weight=0)
    for field in left:
        assert call(a=norm(**bare), **{**left, field: FAKE}) == -1
    assert call(a=norm(weight=0)) == -1
    assert lib.gdn_block_norm_bwd(norm(), None, FAKE, BIG, None) == -1


@pytest.mark.parametrize("T", [1, 63, 64, 65, 4096, 1 << 20, (1 << 31) - (1 << 16)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_no_launch_is_too_large(lib, T, dtype):
    """The workspaces of the largest batches and lengths stay within what the grids hold: sizes are
    finite and grow no faster than the tokens."""
    for B, C in ((1, 8), (1, 1 << 16), (256, 1 << 16), (1 << 20, 16)):
        if B * T > 1 << 36:
            continue
        sc = lib.gdn_gated_scan_bwd_workspace_bytes(scan(B=B, T=T, C=C, dtype=dtype, gate=3, decay=FAKE))
        cv = lib.gdn_short_conv_bwd_workspace_bytes(conv(B=B, T=T, C=C, dtype=dtype))
        assert 0 < sc <= 32 * B * C * (T // 64 + 2) + (1 << 20)
        assert 0 < cv <= 20 * B * C * (T // 64 + 1) + 256
        if C <= 16384:
            nm = lib.gdn_block_norm_bwd_workspace_bytes(norm(B=B, T=T, C=C, dtype=dtype, residual_dtype=dtype))
            assert 0 < nm <= 12 * C * min(B * T, 2048)


def test_binding_refusals():
    import gated_delta_rule_69_amd as gdn
    from gated_delta_rule_69_amd import _block
    x = torch.zeros(1, 4, 16)
    state = torch.zeros(1, 16)
    w = torch.zeros(16, 4)
    for call in (lambda: gdn.gdn_gated_scan_fwd(x, x), lambda: gdn.gdn_gated_scan_step(x, x, state=state),
                 lambda: gdn.gdn_gated_scan_bwd(x, x, d_h=x), lambda: gdn.gdn_short_conv_fwd(x, w),
                 lambda: gdn.gdn_short_conv_step(x, w, state=torch.zeros(1, 3, 16)),
                 lambda: gdn.gdn_short_conv_bwd(x, w, d_y=x), lambda: gdn.gdn_block_norm_fwd(x, x),
                 lambda: gdn.gdn_block_norm_bwd(x, x, d_out=x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    # the packers check before any address is used
    cpu = dict(gate="sigmoid", decay=None, seq_lens=None)
    assert len(_block._scan_args(x, x, None, **cpu)) == ctypes.sizeof(_block.GdnScanArgs)
    for bad, match in ((dict(cpu, gate="tanh"), "unknown gate"), (dict(cpu, gate="power"), "decay"),
                       (dict(cpu, decay=torch.ones(16)), "decay"),
                       (dict(gate="power", decay=torch.ones(8), seq_lens=None), "shape"),
                       (dict(cpu, seq_lens=torch.zeros(1)), "int32")):
        with pytest.raises(ValueError, match=match):
            _block._scan_args(x, x, None, **bad)
    with pytest.raises(ValueError, match="shape"):
        _block._scan_args(x, x[:, :3], None, **cpu)
    with pytest.raises(ValueError, match="must be"):
        _block._scan_args(x, x.double(), None, **cpu)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        _block._scan_args(x.half(), x.half(), None, **cpu)
    with pytest.raises(ValueError, match=r"\[B, T, C\]"):
        _block._scan_args(x[0], x[0], None, **cpu)
    conv_args = lambda **kw: _block._conv_args(x, kw.pop("w", w), **{**dict(bias=None, activation="silu", seq_lens=None, s0=None), **kw})  # noqa: E731
    assert len(conv_args()) == ctypes.sizeof(_block.GdnConvArgs)
    for bad, match in ((dict(activation="gelu"), "activation"), (dict(w=w[0]), "w must be"), (dict(s0=torch.zeros(1, 4, 16)), "shape"),
                       (dict(bias=torch.zeros(8)), "shape"), (dict(w=torch.zeros(4, 16).T), "contiguous")):
        with pytest.raises(ValueError, match=match):
            conv_args(**bad)
    base = dict(gate=None, weight=None, post_norm=False, post_weight=None, scale=None, activation="silu", residual_scale=1.0,
                eps=1e-6, dtype=torch.float32)
    assert len(_block._norm_args(x, x, **base)) == ctypes.sizeof(_block.GdnBlockNormArgs)
    for y, bad, match in ((None, dict(gate=x), "need y"), (None, dict(post_norm=True), "need y"), (x, dict(post_weight=state[0]), "post_norm"),
                          (x, dict(activation="relu"), "activation"), (x, dict(dtype=torch.float16), "residual"),
                          (x, dict(weight=torch.ones(8)), "shape")):
        with pytest.raises(ValueError, match=match):
            _block._norm_args(x, y, **{**base, **bad})
    with pytest.raises(ValueError, match="residual"):
        _block._norm_args(x.bfloat16(), x, **base)


def test_binding_reads_strides_and_refuses_what_it_cannot():
    from gated_delta_rule_69_amd._block import _tokens
    wide = torch.zeros(2, 6, 96)
    view = wide[..., 32:64]
    rows = lambda t: _tokens(t, "x", tuple(t.shape), torch.float32, -1)  # noqa: E731
    assert rows(view) == 96 and rows(view.contiguous()) == 0 and rows(view[:, ::2]) == 192
    assert rows(view[:, :1]) == 6 * 96 and rows(view[:1, :1]) == 0 and rows(view[:, :0]) == 0
    assert rows(view[:1, 1:4]) == 96
    for bad in (view[:, :4], view.transpose(1, 2), view[..., ::2], wide[:, :1].expand(2, 6, 96), view[..., :1].expand(2, 6, 32)):
        with pytest.raises(ValueError, match="strides|shape"):
            rows(bad)
