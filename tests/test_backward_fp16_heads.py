"""fp16 gradients of a sample's K/V head depend on that sample's K/V head alone: large values elsewhere in the batch cost them
no bits."""
import pytest
import torch

import backward_ref as R
import transformer_attention_02_gb300 as ta
from transformer_attention_02_gb300 import attn as A

F16 = torch.float16


def _inputs(B, Hq, Hkv, Sq, Sk, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape):
        return torch.empty(shape, dtype=F16, device="cuda").normal_(generator=g)

    return n(B, Sq, Hq, D).mul_(0.01), n(B, Sq, Hq, D), n(B, Sk, Hkv, D), n(B, Sk, Hkv, D)


def _grads(d_o, q, k, v, **kw):
    o, lse = R.forward(q, k, v, **kw)
    return ta.attention_backward(d_o, q, k, v, o.to(F16), lse.float(), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("shape,causal", [
    ((2, 4, 2, 1000, 1000, 64), False),
    ((2, 4, 2, 1000, 1000, 128), True),
    ((1, 6, 2, 128, 5000, 128), False),              # walks of dQ in parts
    ((1, 16, 2, 900, 300, 64), False),               # walks of dK and dV in parts
    ((40, 8, 8, 260, 300, 64), False),               # more heads than SMs: several for a CTA, one after the other
])
def test_large_values_of_other_heads(shape, causal):
    """One large value of V and one of dO, in the last K/V head. The gradients of the others keep 11 bits: a rounding is off by
    2^-11 / sqrt(3) of the value in the mean square, an operand's and the result's are independent."""
    B, Hq, Hkv, Sq, Sk, D = shape
    d_o, q, k, v = _inputs(*shape, seed=1)
    v[-1, 3, -1, 5] = 60000.0
    d_o[-1, Sq // 2, -1, 7] = 60000.0
    got = _grads(d_o, q, k, v, causal=causal)
    want, _ = R.backward(d_o, q, k, v, causal=causal)
    for name, a, w in zip(("dq", "dk", "dv"), got, want):
        a, w = (t.unflatten(2, (Hkv, t.shape[2] // Hkv)).double() for t in (a, w))
        for b in range(B):
            for h in range(Hkv):
                if (b, h) != (B - 1, Hkv - 1):
                    x, y = a[b, :, h], w[b, :, h]
                    assert float((x - y).norm() / y.norm()) < 2 ** -11 * (2 / 3) ** 0.5, (name, b, h)


@pytest.mark.gpu
@pytest.mark.parametrize("masked", [False, True])
def test_a_sample_by_itself_or_in_a_batch(masked):
    """The same bits (in walks that are not cut, whose sums are added up in one order)."""
    d_o, q, k, v = _inputs(3, 4, 4, 300, 300, 64, seed=2)
    v[1:] *= 1000
    d_o[2] *= 2.0 ** 16
    mask = torch.zeros((3, 300, 300), device="cuda") if masked else None
    kw = dict(causal=True)
    o, lse = ta.attention(q, k, v, mask=mask, **kw)
    whole = ta.attention_backward(d_o, q, k, v, o, lse, mask=mask, **kw)
    for b in range(3):
        s = slice(b, b + 1)
        one = ta.attention_backward(d_o[s], q[s], k[s], v[s], o[s], lse[s], mask=None if mask is None else mask[s], **kw)
        assert all(torch.equal(x, y[s]) for x, y in zip(one, whole)), b


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_infinities_and_nan_set_no_power(value):
    """Of keys before every query's window, whose blocks hold no visible pair."""
    d_o, q, k, v = _inputs(2, 4, 2, 50, 1000, 64, seed=3)
    kw = dict(causal=True, window=20)
    want, bounds = R.backward(d_o, q, k, v, **kw)
    o, lse = R.forward(q, k, v, **kw)
    k[:, :896], v[:, :896] = value, value                        # the first seven blocks of 128
    R.check(ta.attention_backward(d_o, q, k, v, o.to(F16), lse.float(), **kw), want, bounds)


def test_the_workspace_holds_the_words_of_every_head():
    # 320 heads, eight to a block of 64 vectors of 64 values: 200 vectors a head in 7 parts of 4 x 8, a word each behind eight
    # others, in steps of 256 bytes; then two statistics for 128 rows of each head
    assert A.attn_bwd_workspace_bytes(40, 8, 8, 100, 100, 64, 0) == 9216 + 2 * 40 * 8 * 128 * 4
    assert A.attn_bwd_workspace_bytes(1, 1, 1, 100, 100, 64, 0) == 1024 + 2 * 128 * 4
