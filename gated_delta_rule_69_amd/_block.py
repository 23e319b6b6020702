"""ctypes binding of the operators of a block: the gated recurrence a channel, the short
causal convolution before it, and the norms around a block with its gate and residual scale.

Argument marshalling only, as in ``_layer``. Inputs [B, T, C] may be views of one projection's
output: channels contiguous, any distance from token to token. Work runs on the tensors'
device, on its current stream or the given one; what a call allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _layer
from ._layer import (ACTIVATIONS, _beside, _current_stream, _done, _DTYPES, _elsewhere, _f32, _i32, _i64, _io, _on, _packer,
                     _ptr, _refuse, _rows_beside, _whole, _workspace)

SCAN_GATES = {"log": 1, "sigmoid": 2, "power": 3}
SCAN_SPAN = 64


class GdnScanArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("gate", _i32), ("B", _i64), ("T", _i64), ("C", _i64), ("x_stride", _i64),
                ("f_stride", _i64), ("i_stride", _i64), ("x", _ptr), ("f", _ptr), ("i", _ptr), ("decay", _ptr),
                ("seq_lens", _ptr), ("h0", _ptr), ("h_final", _ptr), ("checkpoints", _ptr), ("h", _ptr)]


class GdnScanGrads(ctypes.Structure):
    _fields_ = [("dx", _ptr), ("df", _ptr), ("di", _ptr), ("ddecay", _ptr), ("dh0", _ptr)]


class GdnConvArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("activation", _i32), ("B", _i64), ("T", _i64), ("C", _i64), ("W", _i64),
                ("x_stride", _i64), ("x", _ptr), ("w", _ptr), ("bias", _ptr), ("seq_lens", _ptr), ("s0", _ptr),
                ("s_final", _ptr), ("y", _ptr)]


class GdnConvGrads(ctypes.Structure):
    _fields_ = [("dx", _ptr), ("dw", _ptr), ("dbias", _ptr), ("ds0", _ptr)]


class GdnBlockNormArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("residual_dtype", _i32), ("activation", _i32), ("post_norm", _i32), ("B", _i64),
                ("T", _i64), ("C", _i64), ("r_stride", _i64), ("y_stride", _i64), ("gate_stride", _i64), ("eps", _f32),
                ("residual_scale", _f32), ("r", _ptr), ("y", _ptr), ("gate", _ptr), ("scale", _ptr),
                ("post_weight", _ptr), ("weight", _ptr), ("residual_out", _ptr), ("out", _ptr)]


class GdnBlockNormGrads(ctypes.Structure):
    _fields_ = [("d_residual_out", _ptr), ("d_out", _ptr), ("dr", _ptr), ("dy", _ptr), ("dgate", _ptr), ("dscale", _ptr),
                ("dpost_weight", _ptr), ("dweight", _ptr)]


_scan_pack, _scan_grads_pack = _packer(GdnScanArgs), _packer(GdnScanGrads)
_conv_pack, _conv_grads_pack = _packer(GdnConvArgs), _packer(GdnConvGrads)
_norm_pack, _norm_grads_pack = _packer(GdnBlockNormArgs), _packer(GdnBlockNormGrads)
_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = _layer.load_library()
        size, status = ctypes.c_size_t, ctypes.c_int   # every pointer is untyped: structures come as bytes
        for name, args, res in (
                ("gdn_gated_scan_workspace_bytes", [_ptr], size),
                ("gdn_gated_scan_fwd", [_ptr, _ptr, size, _ptr], status),
                ("gdn_gated_scan_step", [_ptr, _ptr, _ptr], status),
                ("gdn_gated_scan_bwd_workspace_bytes", [_ptr], size),
                ("gdn_gated_scan_bwd", [_ptr, _ptr, _ptr, _ptr, _ptr, size, _ptr], status),
                ("gdn_short_conv_fwd", [_ptr, _ptr], status),
                ("gdn_short_conv_step", [_ptr, _ptr, _ptr], status),
                ("gdn_short_conv_bwd_workspace_bytes", [_ptr], size),
                ("gdn_short_conv_bwd", [_ptr, _ptr, _ptr, _ptr, _ptr, size, _ptr], status),
                ("gdn_block_norm_fwd", [_ptr, _ptr], status),
                ("gdn_block_norm_bwd_workspace_bytes", [_ptr], size),
                ("gdn_block_norm_bwd", [_ptr, _ptr, _ptr, size, _ptr], status)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _lib = lib
    return _lib


# ---- checks ---------------------------------------------------------------------------

def _channels(t, name):
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [B, T, C], got {tuple(shape)}")
    return shape


def _tokens(t, name, shape, dtype, dev):
    """Checks a [B, T, C] tensor that may be a view of a wider one; its token stride (0:
    contiguous)."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return 0
    B, T, C = shape
    sb, st, sc = t.stride()
    ld = st if T > 1 else sb if B > 1 else C
    if (sc != 1 and C > 1) or ld < C or (B > 1 and sb != T * ld):
        raise ValueError(f"{name} must have contiguous channels and sequences T tokens apart, got strides {t.stride()}")
    return ld


def _at(t):
    return 0 if t is None else t.data_ptr()


# ---- the gated recurrence ---------------------------------------------------------------

def _scan_args(x, f, i, gate, decay, seq_lens, h0=None, h_final=0, checkpoints=0, h=0):
    """The arguments as bytes; h_final, checkpoints and h are addresses."""
    dtype, dev = x.dtype, x.get_device()
    io = _io(x, "x")
    B, T, C = shape = _channels(x, "x")
    if gate not in SCAN_GATES:
        raise ValueError(f"unknown gate {gate!r}")
    if (gate == "power") != (decay is not None):
        raise ValueError("decay goes with gate 'power', and only with it")
    f32 = torch.float32
    return _scan_pack(
        io, SCAN_GATES[gate], B, T, C, _tokens(x, "x", shape, dtype, dev), _tokens(f, "f", shape, dtype, dev),
        0 if i is None else _tokens(i, "i", shape, dtype, dev), x.data_ptr(), f.data_ptr(), _at(i),
        _whole(decay, "decay", (C,), f32, dev), _whole(seq_lens, "seq_lens", (B,), torch.int32, dev),
        _whole(h0, "h0", (B, C), f32, dev), h_final, checkpoints, h)


def gdn_gated_scan_fwd(x, f, i=None, *, gate="sigmoid", decay=None, h0=None, h_final=None, h=None, seq_lens=None,
                       workspace=None, stream=None, want_state=True, want_checkpoints=False):
    """The gated recurrence a channel over prompts, h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t, on
    x, f and i [B, T, C] (without ``i`` its factor is 1). ``gate`` says what f is: "log", a = e^f
    (f above 0 grows the state) and m = 1; "sigmoid", a = sigmoid(f) and m = 1 - a; "power",
    a = e^(-decay sigmoid(f)) with a float32 ``decay`` [C] >= 0, and m = sqrt(1 - a^2). Returns (h,
    h_final), allocated when not given; h0 and h_final are float32 [B, C], and h_final may be h0; h
    may be x, f or i where that is contiguous. With ``want_checkpoints`` also the states before
    every 64 tokens, float32 [B, ceil(T / 64), C], which spare the gradients a
    pass over the inputs. ``seq_lens`` [B] int32 gives each sequence's tokens in a padded batch:
    rows of h behind them are left as they are in a given h, and zero in one allocated here."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return gdn_gated_scan_fwd(x, f, i, gate=gate, decay=decay, h0=h0, h_final=h_final, h=h, seq_lens=seq_lens,
                                      workspace=workspace, want_state=want_state, want_checkpoints=want_checkpoints)
    lib = _library()
    B, T, C = shape = _channels(x, "x")
    f32, dev = torch.float32, x.get_device()
    if h is None:
        h = _rows_beside(x, seq_lens)
        to = h.data_ptr()
    else:
        to = _whole(h, "h", shape, x.dtype, dev)
    if h_final is None and want_state:
        h_final = x.new_empty((B, C), dtype=f32)
        after = h_final.data_ptr()
    else:
        after = _whole(h_final, "h_final", (B, C), f32, dev)
    marks = x.new_empty((B, -(-T // SCAN_SPAN), C), dtype=f32) if want_checkpoints else None
    a = _scan_args(x, f, i, gate, decay, seq_lens, h0, after, _at(marks), to)
    ws, at, size = _workspace(workspace, lib.gdn_gated_scan_workspace_bytes(a), "gdn_gated_scan_workspace_bytes", x)
    _done(lib.gdn_gated_scan_fwd(a, at, size, _current_stream(dev)), "gdn_gated_scan_fwd")
    return (h, h_final, marks) if want_checkpoints else (h, h_final)


def gdn_gated_scan_step(x, f, i=None, *, state, gate="sigmoid", decay=None, h=None, seq_lens=None, stream=None):
    """The same recurrence token by token on ``state`` [B, C] (float32, updated in place): T = 1
    is one decode step. Returns h; ``seq_lens`` as above. A sequence of length 0 keeps its state."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return gdn_gated_scan_step(x, f, i, state=state, gate=gate, decay=decay, h=h, seq_lens=seq_lens)
    dev = x.get_device()
    if h is None:
        h = _rows_beside(x, seq_lens)
        to = h.data_ptr()
    else:
        to = _whole(h, "h", x.shape, x.dtype, dev)
    a = _scan_args(x, f, i, gate, decay, seq_lens, state, 0, 0, to)
    _done(_library().gdn_gated_scan_step(a, state.data_ptr(), _current_stream(dev)), "gdn_gated_scan_step")
    return h


def gdn_gated_scan_bwd(x, f, i=None, *, d_h, gate="sigmoid", decay=None, h0=None, dh_final=None, seq_lens=None,
                       checkpoints=None, workspace=None, stream=None):
    """Gradients of (h, h_final) of gdn_gated_scan_fwd for upstream d_h (shape and dtype of h) and
    dh_final (float32 state, optional): {"dx", "df"} and, with ``i``, "di" in the inputs' dtype,
    "dh0" and, for gate "power", "ddecay" in float32. Rows behind a sequence's length are zero.
    ``checkpoints`` are the forward pass's, of the same inputs."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return gdn_gated_scan_bwd(x, f, i, d_h=d_h, gate=gate, decay=decay, h0=h0, dh_final=dh_final,
                                      seq_lens=seq_lens, checkpoints=checkpoints, workspace=workspace)
    lib = _library()
    B, T, C = shape = _channels(x, "x")
    dev, f32 = x.get_device(), torch.float32
    marks = _whole(checkpoints, "checkpoints", (B, -(-T // SCAN_SPAN), C), f32, dev)
    a = _scan_args(x, f, i, gate, decay, seq_lens, h0, 0, marks, 0)
    up, up_state = _whole(d_h, "d_h", shape, x.dtype, dev), _whole(dh_final, "dh_final", (B, C), f32, dev)
    out = {"dx": _beside(x), "df": _beside(x)}
    if i is not None:
        out["di"] = _beside(x)
    if decay is not None:
        out["ddecay"] = _beside(decay)
    out["dh0"] = x.new_empty((B, C), dtype=f32)
    g = _scan_grads_pack(*(_at(out.get(n)) for n in ("dx", "df", "di", "ddecay", "dh0")))
    ws, at, size = _workspace(workspace, lib.gdn_gated_scan_bwd_workspace_bytes(a), "gdn_gated_scan_bwd_workspace_bytes", x)
    _done(lib.gdn_gated_scan_bwd(a, up, up_state, g, at, size, _current_stream(dev)), "gdn_gated_scan_bwd")
    return out


# ---- the short convolution ---------------------------------------------------------------

def _conv_args(x, w, bias, activation, seq_lens, s0, s_final=0, y=0):
    dtype, dev = x.dtype, x.get_device()
    io = _io(x, "x")
    B, T, C = shape = _channels(x, "x")
    if activation not in (None, "silu"):
        raise ValueError(f"unknown activation {activation!r}")
    if w.dim() != 2:
        raise ValueError(f"w must be [C, W], got {tuple(w.shape)}")
    W, f32 = w.shape[1], torch.float32
    return _conv_pack(
        io, ACTIVATIONS["silu"] if activation else 0, B, T, C, W, _tokens(x, "x", shape, dtype, dev), x.data_ptr(),
        _whole(w, "w", (C, W), f32, dev), _whole(bias, "bias", (C,), f32, dev),
        _whole(seq_lens, "seq_lens", (B,), torch.int32, dev), _whole(s0, "s0", (B, W - 1, C), dtype, dev), s_final, y)


def gdn_short_conv_fwd(x, w, bias=None, *, activation="silu", s0=None, s_final=None, y=None, seq_lens=None, stream=None,
                       want_state=True):
    """Causal convolution a channel over the last W tokens, z_t = bias + sum_j w[:, j] x_{t-W+1+j}
    and y = silu(z) ("silu") or z (None): x [B, T, C], float32 w [C, W] (W 2, 3 or 4) and bias [C].
    s0 and s_final [B, W - 1, C] hold the last inputs, oldest first, in x's dtype. Returns (y,
    s_final), allocated when not given; s_final may be s0, and y may be x for up to 8 tokens
    (contiguous; refused for more, whose rows are read again). ``seq_lens`` as for gdn_gated_scan_fwd."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return gdn_short_conv_fwd(x, w, bias, activation=activation, s0=s0, s_final=s_final, y=y, seq_lens=seq_lens,
                                      want_state=want_state)
    B, T, C = shape = _channels(x, "x")
    dev = x.get_device()
    if y is None:
        y = _rows_beside(x, seq_lens)
        to = y.data_ptr()
    else:
        to = _whole(y, "y", shape, x.dtype, dev)
    state = (B, w.shape[-1] - 1, C)
    if s_final is None and want_state:
        s_final = x.new_empty(state)
        after = s_final.data_ptr()
    else:
        after = _whole(s_final, "s_final", state, x.dtype, dev)
    a = _conv_args(x, w, bias, activation, seq_lens, s0, after, to)
    _done(_library().gdn_short_conv_fwd(a, _current_stream(dev)), "gdn_short_conv_fwd")
    return y, s_final


def gdn_short_conv_step(x, w, bias=None, *, state, activation="silu", y=None, seq_lens=None, stream=None):
    """The same with ``state`` [B, W - 1, C] read and replaced: T = 1 is one decode step. Returns
    y, which may be x as above. A sequence of length 0 keeps its state."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return gdn_short_conv_step(x, w, bias, state=state, activation=activation, y=y, seq_lens=seq_lens)
    dev = x.get_device()
    if y is None:
        y = _rows_beside(x, seq_lens)
        to = y.data_ptr()
    else:
        to = _whole(y, "y", x.shape, x.dtype, dev)
    a = _conv_args(x, w, bias, activation, seq_lens, state, 0, to)
    _done(_library().gdn_short_conv_step(a, state.data_ptr(), _current_stream(dev)), "gdn_short_conv_step")
    return y


def gdn_short_conv_bwd(x, w, bias=None, *, d_y, activation="silu", s0=None, ds_final=None, seq_lens=None, workspace=None,
                       stream=None):
    """Gradients of (y, s_final) of gdn_short_conv_fwd for upstream d_y (shape and dtype of y) and
    ds_final (a state, optional): {"dx", "ds0"} in x's dtype, "dw" and, with a bias, "dbias" in
    float32. Rows behind a sequence's length are zero."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return gdn_short_conv_bwd(x, w, bias, d_y=d_y, activation=activation, s0=s0, ds_final=ds_final,
                                      seq_lens=seq_lens, workspace=workspace)
    lib = _library()
    B, T, C = shape = _channels(x, "x")
    dev = x.get_device()
    a = _conv_args(x, w, bias, activation, seq_lens, s0)
    state = (B, w.shape[1] - 1, C)
    up, up_state = _whole(d_y, "d_y", shape, x.dtype, dev), _whole(ds_final, "ds_final", state, x.dtype, dev)
    out = {"dx": _beside(x), "dw": _beside(w), "ds0": x.new_empty(state)}
    if bias is not None:
        out["dbias"] = _beside(bias)
    g = _conv_grads_pack(*(_at(out.get(n)) for n in ("dx", "dw", "dbias", "ds0")))
    ws, at, size = _workspace(workspace, lib.gdn_short_conv_bwd_workspace_bytes(a), "gdn_short_conv_bwd_workspace_bytes", x)
    _done(lib.gdn_short_conv_bwd(a, up, up_state, g, at, size, _current_stream(dev)), "gdn_short_conv_bwd")
    return out


# ---- the norms around a block --------------------------------------------------------------

def _norm_args(residual, y, gate, weight, post_norm, post_weight, scale, activation, residual_scale, eps, dtype,
               residual_out=0, out=0):
    """The arguments as bytes; dtype is that of y, gate and out."""
    rd, dev = residual.dtype, residual.get_device()
    rio = _io(residual, "residual")
    B, T, C = shape = _channels(residual, "residual")
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    if dtype not in _DTYPES or (rd is not torch.float32 and rd is not dtype):
        raise ValueError(f"residual must be float32 or of the type of y and out, got {rd} with {dtype}")
    if y is None and (gate is not None or scale is not None or post_norm):
        raise ValueError("gate, scale and post_norm need y")
    if post_weight is not None and not post_norm:
        raise ValueError("post_weight needs post_norm")
    f32 = torch.float32
    return _norm_pack(
        _DTYPES[dtype], rio, ACTIVATIONS[activation], 1 if post_norm else 0, B, T, C,
        _tokens(residual, "residual", shape, rd, dev), 0 if y is None else _tokens(y, "y", shape, dtype, dev),
        0 if gate is None else _tokens(gate, "gate", shape, dtype, dev), eps, residual_scale, residual.data_ptr(), _at(y),
        _at(gate), _whole(scale, "scale", (C,), f32, dev), _whole(post_weight, "post_weight", (C,), f32, dev),
        _whole(weight, "weight", (C,), f32, dev), residual_out, out)


def gdn_block_norm_fwd(residual, y=None, gate=None, *, weight=None, post_norm=False, post_weight=None, scale=None,
                       activation="sigmoid", residual_scale=1.0, eps=1e-6, residual_out=None, out=None, out_dtype=None,
                       stream=None):
    """What stands between a block's output y and the next block's input: u = y, or its RMS norm
    times post_weight (``post_norm``); residual_out = residual_scale residual + scale
    activation(gate) u; out = the RMS norm of that, before it is rounded, times weight. All
    [B, T, C], weights and scale float32 [C] (None: ones), no gate: factor 1, no y: u = 0.
    The residual is float32 or of y's dtype; out has y's (without y ``out_dtype``, by default the
    residual's). Returns (residual_out, out), which may be residual, y or gate where those are
    contiguous and of the same type."""
    if _elsewhere(residual, "residual", stream):
        with _on(residual, stream):
            return gdn_block_norm_fwd(residual, y, gate, weight=weight, post_norm=post_norm, post_weight=post_weight,
                                      scale=scale, activation=activation, residual_scale=residual_scale, eps=eps,
                                      residual_out=residual_out, out=out, out_dtype=out_dtype)
    dtype = y.dtype if y is not None else out.dtype if out is not None else out_dtype or residual.dtype
    if out_dtype is not None and out_dtype is not dtype:
        raise ValueError(f"out_dtype is {out_dtype}, y or out {dtype}")
    shape, dev = residual.shape, residual.get_device()
    if residual_out is None:
        residual_out = _beside(residual)
        to_r = residual_out.data_ptr()
    else:
        to_r = _whole(residual_out, "residual_out", shape, residual.dtype, dev)
    if out is None:
        like = residual if y is None or residual.dtype is dtype else y
        out = _beside(like) if like.dtype is dtype else residual.new_empty(shape, dtype=dtype)
        to = out.data_ptr()
    else:
        to = _whole(out, "out", shape, dtype, dev)
    a = _norm_args(residual, y, gate, weight, post_norm, post_weight, scale, activation, residual_scale, eps, dtype, to_r, to)
    _done(_library().gdn_block_norm_fwd(a, _current_stream(dev)), "gdn_block_norm_fwd")
    return residual_out, out


def gdn_block_norm_bwd(residual, y=None, gate=None, *, d_out=None, d_residual_out=None, weight=None, post_norm=False,
                       post_weight=None, scale=None, activation="sigmoid", residual_scale=1.0, eps=1e-6, workspace=None,
                       stream=None):
    """Gradients of gdn_block_norm_fwd for upstream d_residual_out (the residual's dtype) and d_out
    (out's), one of which may be None: "dr" in the residual's dtype, "dy" and "dgate" in y's, and
    "dw", "dw_post" and "dscale" in float32, each where its input is given."""
    if _elsewhere(residual, "residual", stream):
        with _on(residual, stream):
            return gdn_block_norm_bwd(residual, y, gate, d_out=d_out, d_residual_out=d_residual_out, weight=weight,
                                      post_norm=post_norm, post_weight=post_weight, scale=scale, activation=activation,
                                      residual_scale=residual_scale, eps=eps, workspace=workspace)
    if d_out is None and d_residual_out is None:
        raise ValueError("d_out or d_residual_out must be given")
    lib = _library()
    dtype = y.dtype if y is not None else d_out.dtype if d_out is not None else residual.dtype
    a = _norm_args(residual, y, gate, weight, post_norm, post_weight, scale, activation, residual_scale, eps, dtype)
    shape, dev = residual.shape, residual.get_device()
    up_r, up = _whole(d_residual_out, "d_residual_out", shape, residual.dtype, dev), _whole(d_out, "d_out", shape, dtype, dev)
    out = {n: _beside(t) for n, t in (("dr", residual), ("dy", y), ("dgate", gate), ("dscale", scale),
                                      ("dw_post", post_weight), ("dw", weight)) if t is not None}
    g = _norm_grads_pack(up_r, up, *(_at(out.get(n)) for n in ("dr", "dy", "dgate", "dscale", "dw_post", "dw")))
    ws, at, size = _workspace(workspace, lib.gdn_block_norm_bwd_workspace_bytes(a), "gdn_block_norm_bwd_workspace_bytes",
                              residual)
    _done(lib.gdn_block_norm_bwd(a, g, at, size, _current_stream(dev)), "gdn_block_norm_bwd")
    return out
