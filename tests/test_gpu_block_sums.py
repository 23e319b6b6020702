"""Weights' gradients as sums over very many sequences."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

B, C = 1 << 18, 8   # a row of partial sums for each sequence: 2^13 one after the other in a thread


def test_conv_weight_sums_of_many_sequences():
    """Equal terms of 1 + 0.9 / 2^12, which float32 sums above 4,096 would drop the end of at every step.
    dz = d_y without activation, so terms are exact; two floats hold a thread's sum, and one rounding of it
    and five of the tree are 6 / 2^24."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev, f64
    term = np.float32(1 + 0.9 / 4096)
    x, d_y = torch.ones((B, 1, C), device=dev()), torch.full((B, 1, C), float(term), device=dev())
    w, bias = torch.ones((C, 2), device=dev()), torch.zeros(C, device=dev())
    g = gdn.gdn_short_conv_bwd(x, w, bias, d_y=d_y, activation=None)
    want = B * float(term)
    for t in (g["dbias"], g["dw"][:, 1]):
        assert np.abs(f64(t) / want - 1).max() < 6 * 2.0 ** -24
    assert (g["dw"][:, 0] == 0).all()


def test_decay_sums_of_many_sequences():
    """Equal terms, -d_h h0 a s with s = 1/2 and decay 1: a term is a product of four roundings, an
    exponential (2^-23) and a sigmoid (two steps); with the sum's six under 2^-20."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev, f64
    zero, h0 = torch.zeros((B, 1, C), device=dev()), torch.full((B, C), 3.3, device=dev())
    d_h = torch.linspace(0.9, 1.1, C).to(dev()).expand(B, 1, C).contiguous()
    g = gdn.gdn_gated_scan_bwd(zero, zero, d_h=d_h, gate="power", decay=torch.ones(C, device=dev()), h0=h0)
    want = -B * f64(d_h[0, 0]) * f64(h0[0]) * np.exp(-0.5) * 0.5
    assert np.abs(f64(g["ddecay"]) / want - 1).max() < 2.0 ** -20


def test_sums_with_an_infinity():
    """An infinite term makes its own column's sum infinite, not NaN."""
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    x, d_y = torch.ones((200, 1, C), device=dev()), torch.ones((200, 1, C), device=dev())
    d_y[40, 0, 3] = float("inf")
    g = gdn.gdn_short_conv_bwd(x, torch.ones((C, 2), device=dev()), torch.zeros(C, device=dev()), d_y=d_y, activation=None)
    assert g["dbias"][3] == float("inf") and (g["dbias"][torch.arange(C, device=dev()) != 3] == 200).all()
