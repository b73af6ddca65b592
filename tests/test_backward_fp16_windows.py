"""Windows and sinks in fp16, whose dS carries powers of two: tiles in whole walks take them back as they are stored, tiles in
parts before the parts are joined, and the two kinds stand side by side where a window's sinks alone are cut."""
import pytest
import torch

import backward_ref as R
import transformer_attention_02_gb300 as ta

F16 = torch.float16


def _case(B, Hq, Hkv, Sq, Sk, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape):
        return torch.empty(shape, dtype=F16, device="cuda").normal_(generator=g)

    d_o, q, k, v = n(B, Sq, Hq, D), n(B, Sq, Hq, D), n(B, Sk, Hkv, D), n(B, Sk, Hkv, D)
    # K/V heads far from one another, each with a power of its own
    far = torch.exp2(torch.arange(B * Hkv, device="cuda").float() % 8 - 5).view(B, 1, Hkv, 1)
    return d_o.mul_(far.repeat_interleave(Hq // Hkv, dim=2).to(F16)), q, k, v.mul_(far.to(F16))


def _check(shape, window, sinks, seed):
    d_o, q, k, v = _case(*shape, seed)
    kw = dict(causal=True, window=window, sinks=sinks)
    o, lse = R.forward(q, k, v, **kw)
    got = ta.attention_backward(d_o, q, k, v, o.to(F16), lse.float(), **kw)
    R.check(got, *R.backward(d_o, q, k, v, **kw))
    again = ta.attention_backward(d_o, q, k, v, o.to(F16), lse.float(), **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("shape,window,sinks", [
    ((1, 2, 1, 300, 300, 64), 1, 0),
    ((1, 2, 2, 700, 700, 128), 100, 4),
    ((2, 2, 1, 1000, 1000, 64), 128, 130),
    ((1, 4, 2, 700, 1500, 128), 333, 0),
    ((1, 2, 2, 1500, 700, 64), 65, 200),
    ((1, 1, 1, 640, 640, 128), 128, 128),
    ((1, 2, 1, 1, 1000, 128), 7, 3),
    ((1, 8, 1, 2000, 2000, 64), 700, 5),
])
def test_windows(shape, window, sinks):
    _check(shape, window, sinks, 21)


@pytest.mark.gpu
@pytest.mark.parametrize("shape,window,sinks", [
    ((1, 8, 1, 2000, 2000, 128), 128, 4),              # a few tiles, the first of them twelve times as long as the others
    ((3, 4, 1, 1000, 1900, 64), 60, 300),              # three blocks of sinks, in each sample
    ((2, 64, 16, 2500, 2500, 64), 100, 130),           # many tiles
])
def test_sinks_that_every_query_sees(shape, window, sinks):
    _check(shape, window, sinks, 22)
