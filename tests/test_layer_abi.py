"""Host-side argument checks of the layer operators: the documented status, before any
launch (no GPU is touched), and the binding's own refusals."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # an aligned, never-dereferenced address
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import os
    from gated_delta_rule_69_amd import _layer, _lib
    if not os.path.exists(_lib.LIB_PATH):
        from gated_delta_rule_69_amd import build
        build.build()
    return _layer._library()


def _fill(a, over):
    for key, val in over.items():
        setattr(a, key, val)
    return a


def linear(**over):
    from gated_delta_rule_69_amd._layer import GdnLinearArgs
    a = GdnLinearArgs(dtype=1, B=2, T=100, H=4, Hk=2, dk=64, dv=64, q=FAKE, k=FAKE, v=FAKE, log_decay=FAKE, o=FAKE)
    return ctypes.byref(_fill(a, over))


def qk(**over):
    from gated_delta_rule_69_amd._layer import GdnQkNormArgs
    a = GdnQkNormArgs(dtype=1, norm=1, B=2, T=100, Hq=4, Hk=2, d=64, rot=32, n_pos=128, eps=1e-6, q_scale=1.0, q=FAKE,
                      k=FAKE, cos=FAKE, sin=FAKE, q_out=FAKE, k_out=2 * FAKE)
    return ctypes.byref(_fill(a, over))


def gated(**over):
    from gated_delta_rule_69_amd._layer import GdnGatedNormArgs
    a = GdnGatedNormArgs(dtype=1, activation=1, B=2, T=100, H=4, d=64, eps=1e-6, x=FAKE, gate=FAKE, y=2 * FAKE)
    return ctypes.byref(_fill(a, over))


LINEAR_SHAPES = [
    ("dtype", 2, -1), ("reserved", 1, -1), ("B", 0, -1), ("T", -1, -1), ("H", 0, -1), ("Hk", 0, -1), ("Hk", 3, -1),
    ("Hk", 8, -1), ("dk", 48, -2), ("dv", 256, -2), ("q_stride", 64, -1), ("k_stride", 132, -1), ("v_stride", 128, -1),
    ("v_stride", 1 << 25, -2), ("B", 1 << 21, -2), ("T", (1 << 31) + 1, -2), ("q_stride", -128, -1),
]
LINEAR_POINTERS = [("q", 0, -1), ("k", 0, -1), ("v", FAKE + 8, -1), ("log_decay", 0, -1), ("log_decay", FAKE + 2, -1),
                   ("seq_lens", FAKE + 1, -1), ("o", 0, -1), ("o", FAKE + 8, -1)]


@pytest.mark.parametrize("field,value,status", LINEAR_SHAPES + LINEAR_POINTERS)
def test_linear_refusals(lib, field, value, status):
    a = linear(**{field: value})
    assert lib.gdn_linear_chunk_fwd(a, FAKE, BIG, None) == status
    assert lib.gdn_linear_recurrent_step(a, FAKE, None) == status
    if (field, value, status) in LINEAR_SHAPES:
        assert lib.gdn_linear_workspace_bytes(a) == 0


def test_linear_workspace_and_state_checks(lib):
    need = lib.gdn_linear_workspace_bytes(linear())
    assert need > 0
    assert lib.gdn_linear_chunk_fwd(linear(), None, 0, None) == -3
    assert lib.gdn_linear_chunk_fwd(linear(), FAKE, need - 1, None) == -3
    assert lib.gdn_linear_chunk_fwd(linear(), FAKE + 16, need, None) == -3
    assert lib.gdn_linear_chunk_fwd(linear(s0=FAKE + 8), FAKE, BIG, None) == -1
    assert lib.gdn_linear_chunk_fwd(linear(s_final=FAKE + 8), FAKE, BIG, None) == -1
    assert lib.gdn_linear_chunk_fwd(None, FAKE, BIG, None) == -1
    assert lib.gdn_linear_recurrent_step(linear(), None, None) == -1
    assert lib.gdn_linear_recurrent_step(linear(), FAKE + 4, None) == -1
    # no tokens: nothing to do without a state to write, and no array is required
    none = dict(T=0, q=0, k=0, v=0, o=0)
    assert lib.gdn_linear_chunk_fwd(linear(**none), FAKE, BIG, None) == 0
    assert lib.gdn_linear_recurrent_step(linear(**none), FAKE, None) == 0


@pytest.mark.parametrize("shape", [dict(dk=128, dv=16), dict(dk=16, dv=128), dict(dk=128, dv=128)])
def test_linear_refuses_more_threads_than_a_launch_has(lib, shape):
    # 2^23 heads of 128 channels would be 2^32 threads; one sequence less is accepted
    a = linear(B=1 << 17, H=64, Hk=64, T=9, **shape)
    grads = (ctypes.c_void_p * 4)(FAKE, FAKE, FAKE, FAKE)
    assert lib.gdn_linear_workspace_bytes(a) == 0 and lib.gdn_linear_bwd_workspace_bytes(a) == 0
    assert lib.gdn_linear_chunk_fwd(a, FAKE, BIG, None) == -2
    assert lib.gdn_linear_recurrent_step(a, FAKE, None) == -2
    assert lib.gdn_linear_chunk_bwd(a, FAKE, None, grads, FAKE, BIG, None) == -2
    a = linear(B=(1 << 17) - 1, H=64, Hk=64, T=9, **shape)
    assert lib.gdn_linear_workspace_bytes(a) > 0 and lib.gdn_linear_bwd_workspace_bytes(a) > 0


def test_linear_backward_checks(lib):
    from gated_delta_rule_69_amd._layer import GdnLinearGrads
    full = dict(dq=FAKE, dk=FAKE, dv=FAKE, ds0=FAKE)
    need = lib.gdn_linear_bwd_workspace_bytes(linear())
    call = lambda a=None, n=need, ws=FAKE, do=FAKE, ds=None, **over: lib.gdn_linear_chunk_bwd(  # noqa: E731
        a or linear(), do, ds, ctypes.byref(GdnLinearGrads(**{**full, **over})), ws, n, None)
    assert need > 0 and lib.gdn_linear_bwd_workspace_bytes(linear(dk=48)) == 0
    assert call(n=need - 1) == -3 and call(ws=None) == -3 and call(ws=FAKE + 16) == -3
    assert call(do=None) == -1 and call(do=FAKE + 2) == -1 and call(ds=FAKE + 8) == -1
    for field in ("dq", "dk", "dv"):
        assert call(**{field: 0}) == -1 and call(**{field: FAKE + 4}) == -1
    assert call(ds0=FAKE + 4) == -1 and call(a=linear(s0=FAKE + 4)) == -1 and call(a=linear(log_decay=0)) == -1
    assert lib.gdn_linear_chunk_bwd(linear(), FAKE, None, None, FAKE, need, None) == -1
    assert call(a=linear(T=0, q=0, k=0, v=0), ds0=0, do=None, dq=0, dk=0, dv=0) == 0


@pytest.mark.parametrize("field,value,status", [
    ("dtype", 3, -1), ("norm", 0, -1), ("norm", 3, -1), ("interleaved", 2, -1), ("eps", -1.0, -1),
    ("eps", float("nan"), -1), ("q_scale", float("inf"), -1), ("B", 0, -1), ("Hq", 0, -1), ("Hk", 0, -1), ("d", 80, -2),
    ("rot", 4, -1), ("rot", 72, -1), ("rot", -8, -1), ("n_pos", 0, -1), ("n_pos", 99, -1), ("q", 0, -1),
    ("k", FAKE + 4, -1), ("cos", 0, -1), ("sin", FAKE + 4, -1), ("q_out", 0, -1), ("k_out", FAKE + 2, -1),
    ("wq", FAKE + 8, -1), ("positions", FAKE + 2, -1), ("q_stride", 250, -1), ("q_stride", 8 * 64 + 4, -1),
    ("reserved", 1, -1),
])
def test_qk_norm_refusals(lib, field, value, status):
    assert lib.gdn_qk_norm_fwd(qk(**{field: value}), None) == status


def test_qk_norm_in_place_needs_contiguous_rows(lib):
    assert lib.gdn_qk_norm_fwd(qk(q_stride=512, q_out=FAKE), None) == -1
    assert lib.gdn_qk_norm_fwd(qk(k_stride=512, k_out=FAKE), None) == -1
    assert lib.gdn_qk_norm_fwd(qk(T=0, q=0, k=0, cos=0, sin=0, q_out=0, k_out=0), None) == 0


def test_qk_norm_backward_refusals(lib):
    from gated_delta_rule_69_amd._layer import GdnQkNormGrads
    full = dict(grad_dtype=1, dq_out=FAKE, dk_out=FAKE, dq=FAKE, dk=FAKE, dwq=FAKE, dwk=FAKE)
    need = lib.gdn_qk_norm_bwd_workspace_bytes(qk())
    call = lambda a=None, n=need, ws=FAKE, **over: lib.gdn_qk_norm_bwd(  # noqa: E731
        a or qk(), ctypes.byref(GdnQkNormGrads(**{**full, **over})), ws, n, None)
    assert need > 0 and lib.gdn_qk_norm_bwd_workspace_bytes(qk(d=48)) == 0
    assert call(n=need - 1) == -3 and call(ws=None) == -3 and call(ws=FAKE + 8) == -3
    for field in ("dq_out", "dk_out", "dq", "dk"):
        assert call(**{field: 0}) == -1 and call(**{field: FAKE + 4}) == -1
    assert call(dwq=FAKE + 2) == -1 and call(grad_dtype=2) == -1 and call(reserved=1) == -1
    assert call(a=qk(dtype=0), grad_dtype=1) == -1
    assert lib.gdn_qk_norm_bwd(qk(), None, FAKE, need, None) == -1


@pytest.mark.parametrize("field,value,status", [
    ("dtype", -1, -1), ("activation", 0, -1), ("activation", 3, -1), ("eps", -1e-9, -1), ("B", 0, -1), ("H", 0, -1),
    ("T", -1, -1), ("d", 24, -2), ("x", 0, -1), ("gate", FAKE + 8, -1), ("weight", FAKE + 4, -1), ("y", 0, -1),
    ("x_stride", 255, -1), ("gate_stride", 260, -1), ("reserved", 7, -1),
])
def test_gated_norm_refusals(lib, field, value, status):
    assert lib.gdn_gated_norm_fwd(gated(**{field: value}), None) == status


def test_gated_norm_in_place_and_backward_refusals(lib):
    from gated_delta_rule_69_amd._layer import GdnGatedNormGrads
    assert lib.gdn_gated_norm_fwd(gated(x_stride=512, y=FAKE), None) == -1
    full = dict(dy=FAKE, dx=FAKE, dgate=FAKE, dweight=FAKE)
    need = lib.gdn_gated_norm_bwd_workspace_bytes(gated())
    call = lambda n=need, ws=FAKE, **over: lib.gdn_gated_norm_bwd(  # noqa: E731
        gated(), ctypes.byref(GdnGatedNormGrads(**{**full, **over})), ws, n, None)
    assert need > 0 and lib.gdn_gated_norm_bwd_workspace_bytes(gated(d=8)) == 0
    assert call(n=need - 1) == -3 and call(ws=FAKE + 128) == -3
    for field in ("dy", "dx", "dgate"):
        assert call(**{field: 0}) == -1
    assert call(dweight=FAKE + 2) == -1
    assert lib.gdn_gated_norm_bwd(gated(), None, FAKE, need, None) == -1


def test_binding_refuses_host_tensors():
    import gated_delta_rule_69_amd as gdn
    x = torch.zeros(1, 4, 2, 16)
    g = torch.zeros(2)
    with pytest.raises(ValueError, match="device tensor"):
        gdn.gdn_linear_chunk_fwd(x, x, x, g)
    with pytest.raises(ValueError, match="device tensor"):
        gdn.gdn_linear_recurrent_step(x, x, x, g, state=torch.zeros(1, 2, 16, 16))
    with pytest.raises(ValueError, match="device tensor"):
        gdn.gdn_qk_norm_fwd(x, x)
    with pytest.raises(ValueError, match="device tensor"):
        gdn.gdn_gated_norm_fwd(x, x)


def test_binding_reads_strides_and_refuses_what_it_cannot():
    """The view checks need no GPU: token strides of a wider tensor pass, others are refused."""
    from gated_delta_rule_69_amd._layer import _rows
    cpu = -1  # the device number of host tensors
    wide = torch.zeros(2, 6, 96)
    view = wide[..., 32:64].unflatten(-1, (2, 16))
    rows = lambda t: _rows(t, "x", tuple(t.shape), torch.float32, cpu)  # noqa: E731
    assert rows(view) == 96
    assert rows(view.contiguous()) == 0                          # contiguous
    assert rows(wide[:1, :4, 32:64].unflatten(-1, (2, 16))) == 96
    assert rows(view[:, :1]) == 6 * 96                           # one token: the stride between sequences
    assert rows(view[:1, :1]) == 0
    assert rows(view[:, :0]) == 0
    assert rows(view[:, ::2]) == 192                             # every second token
    same = wide[:, :1, :32].unflatten(-1, (2, 16)).expand(2, 6, 2, 16)
    for bad in (view[:, :4], view.transpose(1, 2), view[..., ::2], same):
        with pytest.raises(ValueError, match="strides|shape"):
            rows(bad)
    with pytest.raises(ValueError, match="must be"):
        _rows(view.double(), "x", tuple(view.shape), torch.float32, cpu)
