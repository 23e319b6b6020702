"""Inputs of the block operators' GPU tests; tolerances are layer_util.check's: these kernels
too compute in float32 and round once (one step of bf16 is at most 2^-8 of a value)."""
import torch

from layer_util import DTYPES, dev, f64, rand

NAN = float("nan")


def on(t, wide):
    """A [B, T, C] tensor on the device: contiguous, or a view of a wider tensor whose other
    channels are NaN."""
    if t is None:
        return None
    if not wide:
        return t.to(dev())
    B, T, C = t.shape
    big = torch.full((B, T, C + 48), NAN, dtype=t.dtype, device=dev())
    big[..., 16:16 + C] = t.to(dev())
    return big[..., 16:16 + C]


def lengths(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev())


def spoil(t, lens):
    """t with NaN behind each sequence's length: rows that nothing may read."""
    t = t.clone()
    for b, n in enumerate(lens or []):
        t[b, max(n, 0):] = NAN
    return t


def scan_case(B, T, C, dt, gate, igate, seed=0, h0=True, lens=None):
    """Host tensors of a gated scan; gates as a layer's: long and short memories side by side."""
    gen = torch.Generator().manual_seed(seed)
    dtype = DTYPES[dt]
    f = torch.randn((B, T, C), generator=gen, dtype=torch.float64)
    f = -torch.exp(1.5 * f - 2) if gate == "log" else f + 2 if gate == "sigmoid" else f
    case = dict(x=rand(gen, (B, T, C), dtype), f=f.to(dtype), i=rand(gen, (B, T, C), dtype) if igate else None,
                decay=torch.exp(3 * torch.rand(C, generator=gen) - 4).float() if gate == "power" else None,
                h0=rand(gen, (B, C), torch.float32) if h0 else None, d_h=rand(gen, (B, T, C), dtype),
                dh_final=rand(gen, (B, C), torch.float32) if h0 else None)
    return {k: spoil(v, lens) if v is not None and k in ("x", "f", "i", "d_h") else v for k, v in case.items()}


def host(case):
    return {k: None if v is None else f64(v) for k, v in case.items()}
