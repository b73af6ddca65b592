"""8-bit activation checkpoints against PyTorch's own conversions, and the backward pass from them."""
import pytest
import torch

import backward_ref as R
import transformer_attention_02_gb300 as ta
from transformer_attention_02_gb300 import attn as A

BF16, F16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def _power(e):
    """2^e from its bits: computed powers may be off by a bit."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _want(x):
    """(codes, scale): the smallest 2^e >= 2^-100 with max |x| <= 448 * 2^e over the finite values."""
    v = x.double()
    top = torch.where(v.isfinite(), v.abs(), torch.zeros_like(v)).amax(-1)
    e = torch.full_like(top, -100.0)
    for step in (128, 64, 32, 16, 8, 4, 2, 1):                        # the largest e whose scale is too small, and one more
        up = e + step
        e = torch.where(448 * _power(up - 1) < top, up, e)
    scale = _power(e)
    codes = (v / scale[..., None]).clamp(-448, 448).float().to(E4M3)
    return codes, scale.float()


def _same(got, want):
    return torch.equal(got.view(torch.uint8) & 0x7f, want.view(torch.uint8) & 0x7f) and torch.equal(
        got.float().sign().nan_to_num(), want.float().sign().nan_to_num())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,S,H,D", [(1, 1, 1, 64), (2, 333, 8, 64), (1, 77, 3, 128), (4, 1000, 32, 128), (1, 5000, 1, 64)])
def test_codes_scales_and_the_way_back(B, S, H, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(B + S)
    x = torch.empty((B, S, H, D), dtype=dtype, device="cuda").normal_(generator=g)
    x.mul_(torch.exp2(torch.randint(-20, 12, (B, S, H, 1), device="cuda", generator=g).float()).to(dtype))
    codes, scale = ta.checkpoint_store(x)
    want, ws = _want(x)
    assert torch.equal(scale, ws) and _same(codes, want)
    y = ta.checkpoint_load(codes, scale, dtype)
    exact = codes.double() * scale.double()[..., None]
    big = torch.finfo(dtype).max
    assert torch.equal(y, exact.clamp(-big, big).to(dtype))
    # half a step of four significant bits, or of the subnormal codes (2^-9 of the scale), and fp16's own
    err = (y.double() - x.double()).abs()
    assert bool((err <= 2.0 ** -4 * x.double().abs() + (2.0 ** -10 * scale.double())[..., None] + 2.0 ** -25).all())


@pytest.mark.gpu
def test_edges_of_the_scale():
    """Maxima at and next to 448 * 2^e, zeros, the smallest and largest values, infinities and NaN."""
    x = torch.zeros((1, 16, 1, 64), dtype=BF16, device="cuda")
    for i, v in enumerate((448, 450, 446, 1.75, 1.7578125, 3.3895313892515355e38, 2.0 ** -120, 1e-40, 0)):
        x[0, i, 0, 5] = v
        x[0, i, 0, 9] = -v / 3
    x[0, 10, 0, 1], x[0, 10, 0, 2], x[0, 10, 0, 3] = float("inf"), float("-inf"), 2.0
    x[0, 11, 0, 1], x[0, 11, 0, 2] = float("nan"), 3.0
    x[0, 12] = float("inf")
    codes, scale = ta.checkpoint_store(x)
    want, ws = _want(x)
    assert torch.equal(scale, ws) and _same(codes, want)
    assert bool(ta.checkpoint_load(codes, scale)[0, 11, 0, 1].isnan())
    h = torch.full((1, 1, 1, 64), 65504.0, dtype=F16, device="cuda")
    assert bool((ta.checkpoint_load(*ta.checkpoint_store(h), F16) == 65504).all())          # the code says 65536


@pytest.mark.gpu
def test_slices_streams_and_nothing():
    B, S, H, D = 2, 111, 4, 128
    qkv = torch.empty((B, S, 3 * H * D), dtype=BF16, device="cuda").normal_()
    v = qkv[..., 2 * H * D:].unflatten(-1, (H, D))
    a, b = ta.checkpoint_store(v), ta.checkpoint_store(v.contiguous())
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
    back = torch.full_like(qkv, 3.0)
    out = back[..., H * D:2 * H * D].unflatten(-1, (H, D))
    ta.checkpoint_load(*a, out=out)
    assert torch.equal(out, ta.checkpoint_load(*a)) and bool((back[..., :H * D] == 3).all()) and bool((back[..., 2 * H * D:] == 3).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = ta.checkpoint_store(v, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(c[0].view(torch.uint8), a[0].view(torch.uint8))
    empty = ta.checkpoint_store(v[:, :0])
    assert empty[0].shape == (B, 0, H, D) and ta.checkpoint_load(*empty).shape == (B, 0, H, D)


@pytest.mark.gpu
@pytest.mark.parametrize("shape,kw", [
    ((1, 8, 2, 300, 300, 64, BF16), dict(causal=True)),
    ((2, 4, 4, 130, 257, 128, F16), dict()),
    ((1, 4, 1, 500, 500, 128, BF16), dict(causal=True, window=100, sinks=4)),
    ((2, 2, 1, 64, 200, 64, BF16), dict(mask=True)),
    ((1, 2, 1, 1, 1, 64, BF16), dict()),
    ((1, 2, 1, 300, 30, 64, F16), dict(causal=True)),
])
def test_backward_from_checkpoints(shape, kw):
    """Bit for bit the three calls it stands for, and near the formulas at the widened tensors."""
    B, Hq, Hkv, Sq, Sk, D, dtype = shape
    g = torch.Generator(device="cuda").manual_seed(3)
    d_o, q, k, v = (torch.empty(s, dtype=dtype, device="cuda").normal_(generator=g) for s in
                    ((B, Sq, Hq, D), (B, Sq, Hq, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D)))
    if kw.pop("mask", False):
        kw["mask"] = torch.zeros((B, Sq, Sk), device="cuda").masked_fill_(
            torch.rand((B, Sq, Sk), device="cuda", generator=g) < 0.4, float("-inf"))
    q8, k8, v8 = (ta.checkpoint_store(t) for t in (q, k, v))
    got = ta.attention_backward_checkpoint(d_o, q8, k8, v8, **kw)
    q, k, v = (ta.checkpoint_load(*t, dtype) for t in (q8, k8, v8))
    if "window" in kw:
        o, lse = ta.attention_window(q, k, v, window=kw["window"], sinks=kw["sinks"])
    else:
        o, lse = ta.attention(q, k, v, causal=kw.get("causal", False), mask=kw.get("mask"))
    want = ta.attention_backward(d_o, q, k, v, o, lse, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ref, bounds = R.backward(d_o, q, k, v, **kw)
    R.check(got, ref, [2 * b for b in bounds])                 # (o and lse are the forward call's, with P's rounding)


@pytest.mark.gpu
def test_a_training_step_around_the_attention():
    """Packed projection -> positions of two axes -> attention -> checkpoints -> gradients -> back through the positions,
    captured and replayed: the gradient of the packed projection agrees with the same steps one by one."""
    B, S, Hq, Hkv, D, sections = 2, 200, 4, 2, 64, (12, 20)
    parts = (Hq * D, Hkv * D, Hkv * D)
    qkv = torch.empty((B, S, sum(parts)), dtype=BF16, device="cuda").normal_()
    d_o = torch.empty((B, S, Hq, D), dtype=BF16, device="cuda").normal_()
    table = ta.rope_axes_table(64, sections)
    pos = torch.stack([torch.arange(S, device="cuda") // 20, torch.arange(S, device="cuda") % 20], -1).int().expand(B, S, 2).contiguous()

    def split(x):
        return [t.unflatten(-1, (t.shape[-1] // D, D)) for t in x.split(parts, dim=-1)]

    def step():
        q, k, v = split(qkv)
        q, k = ta.rope_axes(q, k, table, pos, sections)
        o, lse = ta.attention(q, k, v.contiguous(), causal=True)
        kept = [ta.checkpoint_store(t) for t in (q, k, v)]
        d_qkv = torch.empty_like(qkv)
        dq, dk, dv = split(d_qkv)
        ta.attention_backward_checkpoint(d_o, *kept, causal=True, dq=dq, dk=dk, dv=dv)
        ta.rope_axes(dq, dk, table, pos, sections, inverse=True, q_out=dq, k_out=dk)
        return o, d_qkv

    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o, d_qkv = step()
    qkv.normal_()
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    assert torch.equal(o, want[0]) and torch.equal(d_qkv, want[1])
    q, k, v = split(qkv)
    q8, k8, v8 = (ta.checkpoint_load(*ta.checkpoint_store(t)) for t in (*ta.rope_axes(q, k, table, pos, sections), v))
    (dq, dk, dv), bounds = R.backward(d_o, q8, k8, v8, causal=True)
    got = split(d_qkv)
    R.check([got[2]], [dv], [2 * bounds[2]])
    for a, w, b, name in ((got[0], dq, bounds[0], "dq"), (got[1], dk, bounds[1], "dk")):
        # turned back in FP32 and rounded once more; a pair's error is at most the sum of both values'
        turned = ta.rope_axes(a.contiguous(), None, table, pos, sections)
        both = (2 * b).unflatten(-1, (D // 2, 2)).sum(-1, keepdim=True).expand(-1, -1, -1, -1, 2).flatten(-2)
        size = w.abs().unflatten(-1, (D // 2, 2)).sum(-1, keepdim=True).expand(-1, -1, -1, -1, 2).flatten(-2)
        assert bool(((turned.double() - w).abs() <= both + 2 * 2.0 ** -8 * (size + both)).all()), name


@pytest.mark.gpu
def test_refusals_of_tensors():
    x = torch.zeros((1, 20, 2, 64), dtype=BF16, device="cuda")
    c = ta.checkpoint_store(x)
    for bad in (lambda: ta.checkpoint_store(x.float()), lambda: ta.checkpoint_store(x.transpose(1, 2)),
                lambda: ta.checkpoint_store(x.cpu()), lambda: ta.checkpoint_store(x, scale=c[1].double()),
                lambda: ta.checkpoint_store(x, codes=x), lambda: ta.checkpoint_load(x, c[1]),
                lambda: ta.checkpoint_load(c[0], c[1][..., :1]), lambda: ta.checkpoint_load(*c, torch.float32),
                lambda: ta.checkpoint_load(*c, F16, out=x), lambda: ta.attention_backward_checkpoint(x.float(), c, c, c),
                lambda: ta.attention_backward_checkpoint(x[:, :5], c, c, c), lambda: ta.attention_backward_checkpoint(x, c, c, (x, c[1])),
                lambda: ta.attention_backward_checkpoint(x, c, c, c, window=4),
                lambda: ta.attention_backward_checkpoint(x, c, c, c, dk=x.half())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ta.AttnError):
        ta.attention_backward_checkpoint(x, c, c, c, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ta.AttnError):
        ta.checkpoint_store(torch.zeros((1, 2, 2, 96), dtype=BF16, device="cuda"))


# ----------------------------------------------------- host checks, no GPU

P = 0x10000


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, 1) for n in ("x", "codes", "scale")], *[({n: P + 8}, 1) for n in ("x", "codes")], (dict(scale=P + 2), 1),
    (dict(stride=120), 1), (dict(stride=132), 1), (dict(B=-1), 1), (dict(S=-1), 1), (dict(H=-1), 1), (dict(D=96), 2), (dict(D=0), 1),
    (dict(B=0), 0), (dict(H=0), 0),
])
def test_refusals_on_the_host(kw, code):
    a = dict(dict(x=P, stride=128, codes=P, scale=P, B=1, S=4, H=2, D=64), **kw)
    for fn in (A.attn_checkpoint_store, A.attn_checkpoint_store_f16):
        assert fn(a["x"], a["stride"], a["codes"], a["scale"], a["B"], a["S"], a["H"], a["D"], None) == code
    for fn in (A.attn_checkpoint_load, A.attn_checkpoint_load_f16):
        assert fn(a["codes"], a["scale"], a["x"], a["stride"], a["B"], a["S"], a["H"], a["D"], None) == code


@pytest.mark.parametrize("fn", [A.attn_bwd_checkpoint, A.attn_bwd_checkpoint_f16])
@pytest.mark.parametrize("kw,code", [
    *[({n: None}, 1) for n in ("g", "q", "k", "v", "qs", "ks", "vs", "dq", "dk", "dv", "ws")],
    *[({n: P + 8}, 1) for n in ("g", "q", "k", "v", "dq", "ws")], (dict(qs=P + 1), 1), (dict(kind=5), 1), (dict(window=2), 1),
    (dict(kind=2), 1), (dict(size=1000), 1), (dict(Hq=3), 1), (dict(D=32), 2), (dict(B=0), 0),
])
def test_backward_refusals_on_the_host(fn, kw, code):
    a = dict(dict(g=P, q=P, k=P, v=P, qs=P, ks=P, vs=P, dq=P, dk=P, dv=P, B=1, Hq=2, Hkv=2, Sq=16, Sk=16, D=64, kind=0, mask=None,
                  window=0, ws=P, size=1 << 20), **kw)
    t = a["D"] * 2
    assert fn(a["g"], a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["dq"], a["dk"], a["dv"], t, t, t, a["B"], a["Hq"], a["Hkv"],
              a["Sq"], a["Sk"], a["D"], 0.0, a["kind"], a["mask"], a["window"], 0, a["ws"], a["size"], None) == code
