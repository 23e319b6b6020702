"""ctypes binding of the operators around the delta rule: linear attention with one decay
a head, the norms of queries and keys with the position rotation, and the gated norm.

Argument marshalling only, as in ``_lib``. q, k, v, x and gate may be views of one
projection's output: heads and channels contiguous, any distance from token to token. Work
runs on the tensors' device, on its current stream or the given one; what a call allocates
belongs to that stream.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from ._lib import DTYPE_BF16, DTYPE_F32, GdnError, load_library

NORMS = {"rms": 1, "l2": 2}
ACTIVATIONS = {"silu": 1, "sigmoid": 2}
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_i32, _i64, _ptr, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class GdnLinearArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("reserved", _i32), ("B", _i64), ("T", _i64), ("H", _i64), ("Hk", _i64),
                ("dk", _i64), ("dv", _i64), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("q", _ptr), ("k", _ptr), ("v", _ptr), ("log_decay", _ptr), ("seq_lens", _ptr),
                ("s0", _ptr), ("s_final", _ptr), ("o", _ptr)]


class GdnLinearGrads(ctypes.Structure):
    _fields_ = [("dq", _ptr), ("dk", _ptr), ("dv", _ptr), ("ds0", _ptr)]


class GdnQkNormArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("norm", _i32), ("B", _i64), ("T", _i64), ("Hq", _i64), ("Hk", _i64),
                ("d", _i64), ("q_stride", _i64), ("k_stride", _i64), ("rot", _i64), ("n_pos", _i64),
                ("interleaved", _i32), ("eps", _f32), ("q_scale", _f32), ("reserved", _i32),
                ("q", _ptr), ("k", _ptr), ("wq", _ptr), ("wk", _ptr), ("cos", _ptr), ("sin", _ptr),
                ("positions", _ptr), ("q_out", _ptr), ("k_out", _ptr)]


class GdnQkNormGrads(ctypes.Structure):
    _fields_ = [("grad_dtype", _i32), ("reserved", _i32), ("dq_out", _ptr), ("dk_out", _ptr),
                ("dq", _ptr), ("dk", _ptr), ("dwq", _ptr), ("dwk", _ptr)]


class GdnGatedNormArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("activation", _i32), ("B", _i64), ("T", _i64), ("H", _i64), ("d", _i64),
                ("x_stride", _i64), ("gate_stride", _i64), ("eps", _f32), ("reserved", _i32),
                ("x", _ptr), ("gate", _ptr), ("weight", _ptr), ("y", _ptr)]


class GdnGatedNormGrads(ctypes.Structure):
    _fields_ = [("dy", _ptr), ("dx", _ptr), ("dgate", _ptr), ("dweight", _ptr)]


def _packer(structure):
    """A function that packs a structure's fields, in order, into bytes: a few times faster
    than filling the ctypes structure, which counts for one decoded token."""
    codes = {_i32: "i", _i64: "q", _ptr: "P", _f32: "f"}
    fmt = struct.Struct("@" + "".join(codes[t] for _, t in structure._fields_))
    assert fmt.size == ctypes.sizeof(structure)
    return fmt.pack


_linear_pack, _linear_grads_pack = _packer(GdnLinearArgs), _packer(GdnLinearGrads)
_qk_pack, _qk_grads_pack = _packer(GdnQkNormArgs), _packer(GdnQkNormGrads)
_gated_pack, _gated_grads_pack = _packer(GdnGatedNormArgs), _packer(GdnGatedNormGrads)
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        size, status = ctypes.c_size_t, ctypes.c_int   # every pointer is untyped: structures come as bytes
        for name, args, res in (
                ("gdn_linear_workspace_bytes", [_ptr], size),
                ("gdn_linear_chunk_fwd", [_ptr, _ptr, size, _ptr], status),
                ("gdn_linear_recurrent_step", [_ptr, _ptr, _ptr], status),
                ("gdn_linear_bwd_workspace_bytes", [_ptr], size),
                ("gdn_linear_chunk_bwd", [_ptr, _ptr, _ptr, _ptr, _ptr, size, _ptr], status),
                ("gdn_qk_norm_fwd", [_ptr, _ptr], status),
                ("gdn_qk_norm_bwd_workspace_bytes", [_ptr], size),
                ("gdn_qk_norm_bwd", [_ptr, _ptr, _ptr, size, _ptr], status),
                ("gdn_gated_norm_fwd", [_ptr, _ptr], status),
                ("gdn_gated_norm_bwd_workspace_bytes", [_ptr], size),
                ("gdn_gated_norm_bwd", [_ptr, _ptr, _ptr, size, _ptr], status)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _lib = lib
    return _lib


def _beside(t):
    """A contiguous tensor of t's shape, type and device (0.6 us less than new_empty takes with
    a shape to parse, of a decoded token's 9)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _rows_beside(v, seq_lens):
    """An output of v's shape. A call writes no rows behind a sequence's length, so those of a
    padded batch are cleared here: whatever the memory held would go on into the next operator,
    and a NaN among it into a weight's gradient."""
    return _beside(v) if seq_lens is None else _beside(v).zero_()


# ---- checks ---------------------------------------------------------------------------

def _elsewhere(t, name, stream):
    """Whether the call has to switch device or stream first; refuses host tensors."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a device tensor")
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, {name} on {t.device}")
        return True
    return dev != _current_device()


def _on(t, stream):
    return torch.cuda.device(t.device) if stream is None else torch.cuda.stream(stream)


def _io(t, name):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}") from None


def _refuse(t, name, shape, dtype, dev):
    """Says what is wrong with a tensor of another device, type or shape."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a device tensor on cuda:{dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t, name, shape, dtype, dev):
    """Checks a [B, T, h, d] tensor that may be a view of a wider one; its token stride (0:
    contiguous)."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return 0
    B, T, h, d = shape
    sb, st, sh, sd = t.stride()
    ld = st if T > 1 else sb if B > 1 else h * d
    if sd != 1 or (h > 1 and sh != d) or ld < h * d or (B > 1 and sb != T * ld):
        raise ValueError(f"{name} must have contiguous heads and sequences T tokens apart, got strides {t.stride()}")
    return ld


def _whole(t, name, shape, dtype, dev):
    """Checks a contiguous tensor; its address (0 for no tensor)."""
    if t is None:
        return 0
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(t, name):
    shape = t.shape
    if len(shape) != 4:
        raise ValueError(f"{name} must be [B, T, heads, d], got {tuple(shape)}")
    return shape


def _workspace(ws, need, where, like):
    """The workspace, its address and its size."""
    if need == 0:
        raise GdnError(-2, where)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif ws.device != like.device or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous device tensor on {like.device}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _done(status, where):
    if status != 0:
        raise GdnError(status, where)


# ---- linear attention -------------------------------------------------------------------

def _linear_args(q, k, v, log_decay, seq_lens, s0, s_final=0, o=0):
    """The arguments as bytes; s_final and o are addresses."""
    dtype, dev = v.dtype, v.get_device()
    io = _io(v, "v")
    B, T, H, dv = rows = _heads(v, "v")
    Hk, dk = _heads(k, "k")[2:]
    key, state, f32 = (B, T, Hk, dk), (B, H, dk, dv), torch.float32
    return _linear_pack(
        io, 0, B, T, H, Hk, dk, dv, _rows(q, "q", key, dtype, dev), _rows(k, "k", key, dtype, dev),
        _rows(v, "v", rows, dtype, dev), q.data_ptr(), k.data_ptr(), v.data_ptr(),
        _whole(log_decay, "log_decay", (H,), f32, dev), _whole(seq_lens, "seq_lens", (B,), torch.int32, dev),
        _whole(s0, "s0", state, f32, dev), s_final, o)


def gdn_linear_chunk_fwd(q, k, v, log_decay, *, s0=None, s_final=None, o=None, seq_lens=None, workspace=None,
                         stream=None, want_state=True):
    """Linear attention over prompts, S_t = e^g S_{t-1} + k_t v_t^T and o_t = S_t^T q_t with a
    constant g <= 0 a value head (``log_decay`` [H]). q, k [B, T, Hk, dk], v [B, T, H, dv], H a
    multiple of Hk. Returns (o, s_final), allocated when not given; s_final may be s0.
    ``seq_lens`` [B] int32 gives each sequence's tokens in a padded batch: rows of o behind
    them are left as they are in a given o, and zero in one allocated here."""
    if _elsewhere(v, "v", stream):
        with _on(v, stream):
            return gdn_linear_chunk_fwd(q, k, v, log_decay, s0=s0, s_final=s_final, o=o, seq_lens=seq_lens,
                                        workspace=workspace, want_state=want_state)
    lib = _library()
    B, _, H, dv = rows = _heads(v, "v")
    state, f32, dev = (B, H, _heads(k, "k")[3], dv), torch.float32, v.get_device()
    if o is None:
        o = _rows_beside(v, seq_lens)
        to = o.data_ptr()
    else:
        to = _whole(o, "o", rows, v.dtype, dev)
    if s_final is None and want_state:
        s_final = v.new_empty(state, dtype=f32)
        after = s_final.data_ptr()
    else:
        after = _whole(s_final, "s_final", state, f32, dev)
    a = _linear_args(q, k, v, log_decay, seq_lens, s0, after, to)
    ws, at, size = _workspace(workspace, lib.gdn_linear_workspace_bytes(a), "gdn_linear_workspace_bytes", v)
    _done(lib.gdn_linear_chunk_fwd(a, at, size, _current_stream(dev)), "gdn_linear_chunk_fwd")
    return o, s_final


def gdn_linear_recurrent_step(q, k, v, log_decay, *, state, o=None, seq_lens=None, stream=None):
    """The same recurrence token by token on ``state`` [B, H, dk, dv] (updated in place):
    T = 1 is one decode step. Returns o; ``seq_lens`` as above. A sequence of length 0 keeps its
    state."""
    if _elsewhere(v, "v", stream):
        with _on(v, stream):
            return gdn_linear_recurrent_step(q, k, v, log_decay, state=state, o=o, seq_lens=seq_lens)
    dev = v.get_device()
    if o is None:
        o = _rows_beside(v, seq_lens)
        to = o.data_ptr()
    else:
        to = _whole(o, "o", v.shape, v.dtype, dev)
    a = _linear_args(q, k, v, log_decay, seq_lens, state, 0, to)
    _done(_library().gdn_linear_recurrent_step(a, state.data_ptr(), _current_stream(dev)), "gdn_linear_recurrent_step")
    return o


def gdn_linear_chunk_bwd(q, k, v, log_decay, *, d_o, s0=None, ds_final=None, seq_lens=None, workspace=None,
                         stream=None):
    """Gradients of (o, s_final) of gdn_linear_chunk_fwd for upstream d_o (shape and dtype of
    o) and ds_final (float32 state, optional): {"dq", "dk", "dv"} in the inputs' dtype and
    "ds0" in float32. Rows behind a sequence's length are zero."""
    if _elsewhere(v, "v", stream):
        with _on(v, stream):
            return gdn_linear_chunk_bwd(q, k, v, log_decay, d_o=d_o, s0=s0, ds_final=ds_final, seq_lens=seq_lens,
                                        workspace=workspace)
    lib = _library()
    a = _linear_args(q, k, v, log_decay, seq_lens, s0)
    dev, f32 = v.get_device(), torch.float32
    state = (v.shape[0], v.shape[2], k.shape[3], v.shape[3])
    up, up_state = _whole(d_o, "d_o", v.shape, v.dtype, dev), _whole(ds_final, "ds_final", state, f32, dev)
    out = {"dq": _beside(q), "dk": _beside(k), "dv": _beside(v),
           "ds0": v.new_empty(state, dtype=f32)}
    g = _linear_grads_pack(*(t.data_ptr() for t in out.values()))
    ws, at, size = _workspace(workspace, lib.gdn_linear_bwd_workspace_bytes(a), "gdn_linear_bwd_workspace_bytes", v)
    _done(lib.gdn_linear_chunk_bwd(a, up, up_state, g, at, size, _current_stream(dev)), "gdn_linear_chunk_bwd")
    return out


# ---- norms of queries and keys -----------------------------------------------------------

def _qk_args(q, k, wq, wk, norm, eps, q_scale, cos, sin, positions, interleaved, q_out, k_out):
    dtype, dev = q.dtype, q.get_device()
    io = _io(q, "q")
    B, T, Hq, d = _heads(q, "q")
    Hk = _heads(k, "k")[2]
    if norm not in NORMS:
        raise ValueError(f"unknown norm {norm!r}")
    rot = n_pos = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos and sin must be [positions, rotated channels / 2]")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        if positions is None and n_pos < T:
            raise ValueError(f"cos and sin have {n_pos} rows for {T} tokens")
    elif positions is not None:
        raise ValueError("positions need cos and sin")
    f32, table, qs, ks = torch.float32, (n_pos, rot // 2), (B, T, Hq, d), (B, T, Hk, d)
    return _qk_pack(
        io, NORMS[norm], B, T, Hq, Hk, d, _rows(q, "q", qs, dtype, dev), _rows(k, "k", ks, dtype, dev), rot, n_pos,
        1 if interleaved else 0, eps, q_scale, 0, q.data_ptr(), k.data_ptr(), _whole(wq, "wq", (d,), f32, dev),
        _whole(wk, "wk", (d,), f32, dev), _whole(cos, "cos", table, f32, dev), _whole(sin, "sin", table, f32, dev),
        _whole(positions, "positions", (B, T), torch.int32, dev), _whole(q_out, "q_out", qs, dtype, dev),
        _whole(k_out, "k_out", ks, dtype, dev))


def gdn_qk_norm_fwd(q, k, wq=None, wk=None, *, norm="rms", eps=1e-6, q_scale=1.0, cos=None, sin=None,
                    positions=None, interleaved=False, q_out=None, k_out=None, stream=None):
    """Norm of each head's query and key ("rms" or "l2", float32 weights [d]), rotation of
    the first 2 * cos.shape[1] channels by the token's position (rows of the float32 tables
    cos, sin; ``positions`` [B, T] int32, default 0 .. T-1), and q_scale on queries. q [B, T,
    Hq, d], k [B, T, Hk, d]. Returns (q_out, k_out); they may be q and k where those are
    contiguous. A position outside the tables gives a row of NaN."""
    if _elsewhere(q, "q", stream):
        with _on(q, stream):
            return gdn_qk_norm_fwd(q, k, wq, wk, norm=norm, eps=eps, q_scale=q_scale, cos=cos, sin=sin,
                                   positions=positions, interleaved=interleaved, q_out=q_out, k_out=k_out)
    if q_out is None:
        q_out = _beside(q)
    if k_out is None:
        k_out = q.new_empty(k.shape)
    a = _qk_args(q, k, wq, wk, norm, eps, q_scale, cos, sin, positions, interleaved, q_out, k_out)
    _done(_library().gdn_qk_norm_fwd(a, _current_stream(q.get_device())), "gdn_qk_norm_fwd")
    return q_out, k_out


def gdn_qk_norm_bwd(q, k, wq=None, wk=None, *, dq_out, dk_out, norm="rms", eps=1e-6, q_scale=1.0, cos=None,
                    sin=None, positions=None, interleaved=False, workspace=None, stream=None):
    """Gradients of gdn_qk_norm_fwd: {"dq", "dk"} in the inputs' dtype, and {"dwq", "dwk"}
    (float32) where the weights are given. dq_out and dk_out are contiguous, in the inputs'
    dtype or both float32."""
    if _elsewhere(q, "q", stream):
        with _on(q, stream):
            return gdn_qk_norm_bwd(q, k, wq, wk, dq_out=dq_out, dk_out=dk_out, norm=norm, eps=eps, q_scale=q_scale,
                                   cos=cos, sin=sin, positions=positions, interleaved=interleaved, workspace=workspace)
    lib = _library()
    a = _qk_args(q, k, wq, wk, norm, eps, q_scale, cos, sin, positions, interleaved, None, None)
    dev = q.get_device()
    up = dq_out.dtype if dq_out.dtype is torch.float32 else q.dtype
    uq, uk = _whole(dq_out, "dq_out", q.shape, up, dev), _whole(dk_out, "dk_out", k.shape, up, dev)
    out = {"dq": _beside(q), "dk": _beside(k)}
    for name, w in (("dwq", wq), ("dwk", wk)):
        if w is not None:
            out[name] = _beside(w)
    at = {n: t.data_ptr() for n, t in out.items()}
    g = _qk_grads_pack(_DTYPES[up], 0, uq, uk, at["dq"], at["dk"], at.get("dwq", 0), at.get("dwk", 0))
    ws, wp, size = _workspace(workspace, lib.gdn_qk_norm_bwd_workspace_bytes(a), "gdn_qk_norm_bwd_workspace_bytes", q)
    _done(lib.gdn_qk_norm_bwd(a, g, wp, size, _current_stream(dev)), "gdn_qk_norm_bwd")
    return out


# ---- gated norm ----------------------------------------------------------------------------

def _gated_args(x, gate, weight, eps, activation, out):
    dtype, dev = x.dtype, x.get_device()
    io = _io(x, "x")
    B, T, H, d = shape = _heads(x, "x")
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    return _gated_pack(
        io, ACTIVATIONS[activation], B, T, H, d, _rows(x, "x", shape, dtype, dev),
        _rows(gate, "gate", shape, dtype, dev), eps, 0, x.data_ptr(), gate.data_ptr(),
        _whole(weight, "weight", (d,), torch.float32, dev), _whole(out, "out", shape, dtype, dev))


def gdn_gated_norm_fwd(x, gate, weight=None, *, eps=1e-6, activation="silu", out=None, stream=None):
    """RMS norm of each head's output times ``activation`` ("silu" or "sigmoid") of its gate:
    x, gate [B, T, H, d], weight [d] float32. Returns out, which may be x or gate where that
    is contiguous."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return gdn_gated_norm_fwd(x, gate, weight, eps=eps, activation=activation, out=out)
    if out is None:
        out = _beside(x)
    a = _gated_args(x, gate, weight, eps, activation, out)
    _done(_library().gdn_gated_norm_fwd(a, _current_stream(x.get_device())), "gdn_gated_norm_fwd")
    return out


def gdn_gated_norm_bwd(x, gate, weight=None, *, d_out, eps=1e-6, activation="silu", workspace=None, stream=None):
    """Gradients of gdn_gated_norm_fwd: {"dx", "dgate"} in the inputs' dtype, and "dw"
    (float32) where the weight is given."""
    if _elsewhere(x, "x", stream):
        with _on(x, stream):
            return gdn_gated_norm_bwd(x, gate, weight, d_out=d_out, eps=eps, activation=activation, workspace=workspace)
    lib = _library()
    a = _gated_args(x, gate, weight, eps, activation, None)
    dev = x.get_device()
    up = _whole(d_out, "d_out", x.shape, x.dtype, dev)
    out = {"dx": _beside(x), "dgate": _beside(x)}
    if weight is not None:
        out["dw"] = _beside(weight)
    g = _gated_grads_pack(up, out["dx"].data_ptr(), out["dgate"].data_ptr(), 0 if weight is None else out["dw"].data_ptr())
    ws, at, size = _workspace(workspace, lib.gdn_gated_norm_bwd_workspace_bytes(a), "gdn_gated_norm_bwd_workspace_bytes", x)
    _done(lib.gdn_gated_norm_bwd(a, g, at, size, _current_stream(dev)), "gdn_gated_norm_bwd")
    return out
