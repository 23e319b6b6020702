"""MI355X (gfx950) forward pass of the fine-grained gated delta rule (FG2-GDN) and
its KDA, GDN, DeltaProduct and GDN2/RWKV-7-style variants, and the operators of a layer
around it: linear attention with one decay a head, the norms of queries and keys with the
position rotation, and the gated norm of outputs; and those of a block: the gated recurrence
a channel, the short convolution and the norms around it.

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
_BLOCK = ("gdn_gated_scan_fwd", "gdn_gated_scan_step", "gdn_gated_scan_bwd", "gdn_short_conv_fwd", "gdn_short_conv_step",
          "gdn_short_conv_bwd", "gdn_block_norm_fwd", "gdn_block_norm_bwd")


def __getattr__(name):  # the layer's and the block's bindings need torch at import; the rest does not
    if name in _LAYER:
        from . import _layer as module
        names = _LAYER
    elif name in _BLOCK:
        from . import _block as module
        names = _BLOCK
    else:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    for n in names:
        globals()[n] = getattr(module, n)
    return globals()[name]
