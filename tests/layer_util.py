"""Inputs and tolerances of the layer operators' GPU tests.

Tolerances. The kernels compute in float32 (matrix products of bf16 inputs carry their
second factor as sums of bf16 parts, to 2^-16 for values that end in bf16 and to 2^-24 for
float32 results) and round once. So a bf16 output is off by at most half a step, 2^-8 of
its value, plus an inner error that these sizes keep under 2^-11 of the tensor's norm; a
float32 output is held to rel-L2 1e-5 and normwise 1e-4, as the recurrence's float32
results are: sums of a few hundred terms at 2^-24 each, 200 * 2^-24 = 1.2e-5 in the worst
case and its square root's share in practice.
"""
import numpy as np
import torch

import oracle

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev():
    return torch.device("cuda:0")


def rand(gen, shape, dtype, scale=1.0):
    """A CPU tensor of N(0, scale^2) in ``dtype``."""
    return (torch.randn(shape, generator=gen, dtype=torch.float64) * scale).to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(got, want, name, exact_rows=None):
    """``got`` (device tensor) against ``want`` (float64 array) by the rule above."""
    x = f64(got)
    want = np.asarray(want, dtype=np.float64)
    assert x.shape == want.shape, (name, x.shape, want.shape)
    assert np.isfinite(x).all(), f"{name}: not finite"
    l2, top = (2.0 ** -8 + 2.0 ** -11,) * 2 if got.dtype == torch.bfloat16 else (1e-5, 1e-4)
    e, m = oracle.rel_l2(x, want), oracle.max_rel(x, want)
    assert e <= l2 and m <= top, f"{name}: rel-L2 {e:.2e} (at most {l2:.2e}), normwise {m:.2e} (at most {top:.2e})"


def fused(parts):
    """The same [B, T, h, d] tensors as views of one wider tensor, on the device."""
    B, T = parts[0].shape[:2]
    x = torch.cat([p.reshape(B, T, -1) for p in parts], -1).to(dev())
    out = torch.split(x, [p.shape[2] * p.shape[3] for p in parts], -1)
    return [o.unflatten(-1, p.shape[2:]) for o, p in zip(out, parts)]
