"""Block operators whose outputs take the place of an input: bit for bit what they give apart, or refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _conv_case(B, T, C, dt, seed=1):
    from layer_util import DTYPES, dev, rand
    gen = torch.Generator().manual_seed(seed)
    return (rand(gen, (B, T, C), DTYPES[dt]).to(dev()), rand(gen, (C, 4), torch.float32, 0.5).to(dev()),
            rand(gen, (B, 3, C), DTYPES[dt]).to(dev()))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,lens", [(1, 1, 8, None), (3, 2, 264, None), (5, 8, 520, [8, 0, 3, 1, 7]), (1030, 8, 8, None),
                                        (600, 5, 1024, None)])
def test_conv_of_few_tokens_in_place(B, T, C, lens, dt):
    import gated_delta_rule_69_amd as gdn
    from block_util import lengths
    x, w, s0 = _conv_case(B, T, C, dt)
    kw = dict(seq_lens=lengths(lens))
    y, end = gdn.gdn_short_conv_fwd(x, w, s0=s0, **kw)
    for step in (False, True):
        own, state = x.clone(), s0.clone()
        if step:
            got = gdn.gdn_short_conv_step(own, w, state=state, y=own, **kw)
        else:
            got, _ = gdn.gdn_short_conv_fwd(own, w, s0=state, s_final=state, y=own, **kw)
        assert got is own and torch.equal(state, end)
        for b in range(B if lens else 0):
            assert torch.equal(own[b, lens[b]:], x[b, lens[b]:])
            own[b, lens[b]:] = 0
        assert torch.equal(own, y)


def test_conv_of_more_tokens_is_refused_in_place():
    import gated_delta_rule_69_amd as gdn
    from layer_util import dev
    x, w, s0 = _conv_case(2, 9, 16, "f32")
    keep = x.clone()
    for call in (lambda: gdn.gdn_short_conv_fwd(x, w, y=x), lambda: gdn.gdn_short_conv_step(x, w, state=s0, y=x)):
        with pytest.raises(gdn.GdnError):
            call()
    assert torch.equal(x, keep)
    # between the rows of a view there is room
    big = torch.zeros(8 * 512, device=dev())
    view, room = big.as_strided((1, 7, 64), (7 * 512, 512, 1)), big[64:512].view(1, 7, 64)
    x, w, _ = _conv_case(1, 7, 64, "f32")
    view.copy_(x)
    y, _ = gdn.gdn_short_conv_fwd(view, w, y=room)
    assert y is room and torch.equal(y, gdn.gdn_short_conv_fwd(x, w)[0]) and torch.equal(view, x)
