"""MI355X (gfx950) forward pass of the fine-grained gated delta rule (FG2-GDN) and
its KDA, GDN, DeltaProduct and GDN2/RWKV-7-style variants, and the operators of a layer
around it: linear attention with one decay a head, the norms of queries and keys with the
position rotation, and the gated norm of outputs.

The computation lives in libgdn.so (hand-written HIP kernels behind the C ABI of
include/gdn.h); this package is its ctypes binding.
"""
from ._lib import (GdnArgs, GdnError, VARIANTS, gdn_abi_version, gdn_asym_stabilize,  # noqa: F401
                   gdn_chunk_fwd, gdn_chunk_fwd_args, gdn_chunk_fwd_static, gdn_chunk_prepare, gdn_chunk_scan, gdn_final_state,
                   gdn_recurrent_bwd, gdn_recurrent_step, gdn_status_str, gdn_workspace_bytes,
                   load_library,
                   make_args)

_LAYER = ("gdn_linear_chunk_fwd", "gdn_linear_recurrent_step", "gdn_linear_chunk_bwd", "gdn_qk_norm_fwd",
          "gdn_qk_norm_bwd", "gdn_gated_norm_fwd", "gdn_gated_norm_bwd")


def __getattr__(name):  # the layer's binding needs torch at import; the rest does not
    if name not in _LAYER:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from . import _layer
    for n in _LAYER:
        globals()[n] = getattr(_layer, n)
    return globals()[name]
