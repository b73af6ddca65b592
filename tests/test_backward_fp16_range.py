"""fp16 gradients that the type holds, from dS that it does not: dS is carried times a power of two, up or down.

Bounds: those of backward_ref.py and, where the power s is below zero, half a step of the subnormal range taken back by it,
2^-25 / 2^s for each dS of a visible pair.
"""
import math

import pytest
import torch

import backward_ref as R
import transformer_attention_02_gb300 as ta
from transformer_attention_02_gb300 import attn as A

F16 = torch.float16


def _normal(shapes, sizes, seed, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed)
    return [torch.empty(s, dtype=F16, device=dev).normal_(generator=g).mul_(f) for s, f in zip(shapes, sizes)]


def _want(d_o, q, k, v, *, causal=False, mask=None, window=0, sinks=0, scale=None):
    """(gradients, bounds) in FP64, for any power that keeps 2 D max|dO| max|V| at or below 2^15 (one step to spare)."""
    want, bounds = R.backward(d_o, q, k, v, causal=causal, mask=mask, window=window, sinks=sinks, scale=scale)
    D, G = q.shape[3], q.shape[2] // k.shape[2]
    above = math.log2(max(2 * D * float(d_o.abs().max()) * float(v.abs().max()), 2.0 ** -40))
    step = 2.0 ** (-25 + max(0, math.floor(above) + 2 - 15))
    see = R.visible(q.shape[1], k.shape[1], causal, window, sinks, q.device).double() * step * (scale or 1 / math.sqrt(D))
    kk = k.double().abs().repeat_interleave(G, dim=2)
    e_dq = torch.einsum("ij,bjhd->bihd", see, kk)
    e_dk = torch.einsum("ij,bihd->bjhd", see, q.double().abs()).unflatten(2, (k.shape[2], G)).sum(3)
    return want, (bounds[0] + 1.01 * e_dq, bounds[1] + 1.01 * e_dk, bounds[2])


def _check(got, want, bounds, label=""):
    """Within the bound wherever the gradient and its bound fit the type."""
    torch.cuda.synchronize()
    assert A.attn_last_status(torch.cuda.current_stream().cuda_stream) == A.ATTN_OK
    for name, a, w, b in zip(("dq", "dk", "dv"), got, want, bounds):
        fits = w.abs() + b < torch.finfo(F16).max
        assert bool(torch.isfinite(a[fits]).all()), f"{label} {name}: not finite"
        err = ((a.double() - w).abs() - b)[fits]
        assert bool((err <= 0).all()), f"{label} {name}: {float(err.max()):.3e} past the bound"


def _ds_max(d_o, q, k, v, causal):
    """The largest |dS| of the formulas."""
    o, lse = R.forward(q, k, v, causal=causal)
    G = q.shape[2] // k.shape[2]
    kk, vv = (t.double().repeat_interleave(G, dim=2) for t in (k, v))
    z = torch.einsum("bihd,bjhd->bhij", q.double(), kk) / math.sqrt(q.shape[3])
    p = (z - lse[..., None]).exp().masked_fill(~R.visible(q.shape[1], k.shape[1], causal, device=q.device), 0.0)
    dp = torch.einsum("bihd,bjhd->bhij", d_o.double(), vv) - (d_o.double() * o).sum(-1).transpose(1, 2)[..., None]
    return float((p * dp).abs().max())


def _grads(d_o, q, k, v, **kw):
    o, lse = R.forward(q, k, v, **kw)
    return ta.attention_backward(d_o, q, k, v, o.to(F16), lse.float(), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("masked", [False, True])
def test_one_query_of_two_far_values(masked):
    """By hand: dP = +-256 * 64 * 10, P near 1/2, so that dS is near +-81920; the gradients are a few thousand."""
    q = torch.full((1, 1, 1, 64), 0.5, dtype=F16, device="cuda")
    k = torch.full((1, 2, 1, 64), 0.1, dtype=F16, device="cuda")
    k[0, 1] = 0.0996
    v = torch.full((1, 2, 1, 64), 10.0, dtype=F16, device="cuda")
    v[0, 1] = -10.0
    d_o = torch.full_like(q, 256.0)
    kw = dict(mask=torch.zeros((1, 1, 2), device="cuda")) if masked else {}
    want, bounds = _want(d_o, q, k, v, **kw)
    assert _ds_max(d_o, q, k, v, False) > 65504 and max(float(w.abs().max()) for w in want) < 6000
    _check(_grads(d_o, q, k, v, **kw), want, bounds)


@pytest.mark.gpu
@pytest.mark.parametrize("shape,sizes,seed", [
    ((1, 1, 1, 2048, 2048, 128), (3000.0, 2.0, 1.0, 3.0), 1),
    ((1, 4, 4, 200, 200, 128), (4000.0, 1.0, 1.0, 4.0), 2),
    ((1, 8, 2, 300, 300, 64), (4000.0, 1.0, 1.0, 8.0), 3),
])
def test_gradients_of_a_scaled_loss(shape, sizes, seed):
    B, Hq, Hkv, Sq, Sk, D = shape
    d_o, q, k, v = _normal([(B, Sq, Hq, D), (B, Sq, Hq, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D)], sizes, seed)
    want, bounds = _want(d_o, q, k, v, causal=True)
    assert _ds_max(d_o, q, k, v, True) > 65504
    _check(_grads(d_o, q, k, v, causal=True), want, bounds, str(shape))


@pytest.mark.gpu
@pytest.mark.parametrize("causal,masked", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("d_o_size,v_size", [(2.0 ** -20, 1.0), (1.0, 1.0), (60000.0, 2.0 ** -10), (60000.0, 1.0), (60000.0, 100.0),
                                             (1.0, 60000.0), (2.0 ** -10, 60000.0)])
def test_up_to_the_largest_values(d_o_size, v_size, causal, masked):
    """dO and V uniform up to the type's largest values: a gradient that the type holds comes out, whatever dS is."""
    g = torch.Generator(device="cuda").manual_seed(4)
    shapes = [(2, 260, 4, 64), (2, 260, 4, 64), (2, 260, 2, 64), (2, 260, 2, 64)]
    d_o, q, k, v = (torch.empty(s, device="cuda").uniform_(-f, f, generator=g).to(F16)
                    for s, f in zip(shapes, (d_o_size, 1.0, 2.0 ** -6, v_size)))
    kw = dict(causal=causal)
    if masked:
        kw["mask"] = torch.zeros((2, 260, 260), device="cuda").masked_fill_(
            torch.rand((2, 260, 260), device="cuda", generator=g) < 0.3, float("-inf"))
    want, bounds = _want(d_o, q, k, v, **kw)
    _check(_grads(d_o, q, k, v, **kw), want, bounds)


@pytest.mark.gpu
def test_from_checkpoints():
    """The same from 8-bit checkpoints, whose forward pass is the framework's own."""
    d_o, q, k, v = _normal([(1, 200, 4, 128)] * 4, (4000.0, 1.0, 1.0, 4.0), 5)
    kept = [ta.checkpoint_store(t) for t in (q, k, v)]
    got = ta.attention_backward_checkpoint(d_o, *kept, causal=True)
    q, k, v = (ta.checkpoint_load(*t, F16) for t in kept)
    want, bounds = _want(d_o, q, k, v, causal=True)
    assert _ds_max(d_o, q, k, v, True) > 65504
    # (o and lse are the forward call's, with P's rounding: delta by that much again)
    _check(got, want, [2 * b for b in bounds])


@pytest.mark.gpu
@pytest.mark.parametrize("shape,kw", [
    ((1, 8, 1, 1500, 1500, 64), dict(causal=True)),                          # walks of both kernels in parts
    ((1, 1, 1, 40, 6000, 128), dict()),
    ((1, 16, 1, 700, 100, 64), dict(causal=False)),
    ((1, 8, 1, 2000, 2000, 128), dict(causal=True, window=128, sinks=4)),     # the sinks' tiles in parts, the others whole
    ((2, 16, 8, 600, 600, 64), dict(causal=True, window=100, sinks=0)),
])
def test_in_parts_and_windows(shape, kw):
    """Powers below zero, taken back before the parts are joined or as a tile is stored."""
    B, Hq, Hkv, Sq, Sk, D = shape
    d_o, q, k, v = _normal([(B, Sq, Hq, D), (B, Sq, Hq, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D)], (3000.0, 1.0, 1.0, 30.0), 6)
    want, bounds = _want(d_o, q, k, v, **kw)
    got = _grads(d_o, q, k, v, **kw)
    _check(got, want, bounds, str(shape))
    again = _grads(d_o, q, k, v, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
