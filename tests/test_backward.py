"""Gradients of the attention against the formulas in 64 bits (backward_ref.py)."""
import pytest
import torch

import backward_ref as R
import transformer_attention_02_gb300 as ta
from transformer_attention_02_gb300 import attn as A

BF16, F16 = torch.bfloat16, torch.float16


def _inputs(B, Hq, Hkv, Sq, Sk, D, dtype, seed=0, dev="cuda", size=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)

    def n(*shape):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)

    return n(B, Sq, Hq, D).mul_(size), n(B, Sq, Hq, D), n(B, Sk, Hkv, D), n(B, Sk, Hkv, D)


def _run(d_o, q, k, v, *, mask=None, **kw):
    o, lse = R.forward(q, k, v, mask=mask, **kw)
    got = ta.attention_backward(d_o, q, k, v, o.to(q.dtype), lse.float(), mask=mask, **kw)
    torch.cuda.synchronize()
    assert A.attn_last_status(torch.cuda.current_stream().cuda_stream) == A.ATTN_OK
    return got


def _check(d_o, q, k, v, label="", **kw):
    got = _run(d_o, q, k, v, **kw)
    R.check(got, *R.backward(d_o, q, k, v, **kw), label)
    return got


def test_the_formulas_agree_with_differences():
    """The 64-bit reference itself, against central differences of sum(dO o O): h^2 times a third derivative of order 1."""
    g = torch.Generator().manual_seed(1)
    q, k, v, d_o = (torch.randn(1, n, h, 8, generator=g, dtype=torch.float64) for n, h in ((5, 4), (7, 2), (7, 2), (5, 4)))
    q, k, v = (t.to(torch.float64) for t in (q, k, v))
    mask = torch.zeros(1, 5, 7)
    mask[0, 1, 3] = float("-inf")
    mask[0, 2] = float("-inf")
    for kw in (dict(), dict(causal=True), dict(causal=True, window=2, sinks=1), dict(mask=mask), dict(mask=mask, causal=True)):
        (dq, dk, dv), _ = R.backward(d_o, q, k, v, **kw)
        h = 1e-5
        for x, dx in ((q, dq), (k, dk), (v, dv)):
            for at in ((0, 0, 0, 0), (0, 2, 1, 3), (0, x.shape[1] - 1, x.shape[2] - 1, 7)):
                val = []
                for s in (h, -h):
                    old = x[at].item()
                    x[at] = old + s
                    val.append(float((R.forward(q, k, v, **kw)[0] * d_o).sum()))
                    x[at] = old
                assert abs((val[0] - val[1]) / (2 * h) - float(dx[at])) < 1e-7


SHAPES = [
    # B, Hq, Hkv, Sq, Sk, D
    (1, 1, 1, 128, 128, 128),
    (1, 2, 2, 128, 128, 64),
    (2, 4, 2, 100, 100, 64),
    (1, 1, 1, 1, 1, 128),
    (1, 3, 1, 1, 300, 128),
    (2, 2, 1, 300, 1, 64),
    (2, 7, 1, 129, 385, 128),
    (1, 4, 2, 513, 257, 128),
    (3, 2, 2, 255, 640, 64),
    (1, 8, 2, 700, 700, 128),
    (2, 40, 40, 130, 259, 64),
    (1, 2, 2, 2000, 2100, 128),
    # few tiles, long walks: cut into parts whose sums are joined
    (1, 8, 1, 1500, 1500, 64),
    (1, 1, 1, 40, 6000, 128),
    (1, 16, 1, 700, 100, 64),
    (2, 3, 1, 1, 3000, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(shape, causal, dtype):
    _check(*_inputs(*shape, dtype), causal=causal, label=str(shape))


@pytest.mark.gpu
@pytest.mark.parametrize("shape,window,sinks", [
    ((1, 2, 1, 300, 300, 64), 1, 0),
    ((1, 2, 2, 700, 700, 128), 100, 4),
    ((2, 2, 1, 1000, 1000, 64), 128, 130),
    ((1, 4, 2, 700, 1500, 128), 333, 0),
    ((1, 2, 2, 1500, 700, 64), 65, 200),
    ((1, 1, 1, 640, 640, 128), 128, 128),
    ((1, 2, 1, 400, 400, 128), 10 ** 12, 10 ** 12),
    ((1, 2, 1, 1, 1000, 128), 7, 3),
    ((1, 8, 1, 2000, 2000, 64), 700, 5),
])
def test_windows(shape, window, sinks):
    w = dict(causal=True, window=min(window, 1 << 30), sinks=min(sinks, 1 << 30))
    d_o, q, k, v = _inputs(*shape, BF16, seed=3)
    o, lse = R.forward(q, k, v, **w)
    got = ta.attention_backward(d_o, q, k, v, o.to(BF16), lse.float(), causal=True, window=window, sinks=sinks)
    R.check(got, *R.backward(d_o, q, k, v, **w))


@pytest.mark.gpu
@pytest.mark.parametrize("shape,window,sinks", [
    ((1, 8, 1, 2000, 2000, 128), 128, 4),              # a few tiles, the first of them twelve times as long as the others
    ((3, 4, 1, 1000, 1900, 64), 60, 300),              # three blocks of sinks, in each sample
    ((2, 64, 16, 2500, 2500, 64), 100, 130),           # many tiles
])
def test_sinks_that_every_query_sees(shape, window, sinks):
    """The keys of the sinks take part in every query's sum: their tiles' walks are cut, and joined, apart from the others."""
    d_o, q, k, v = _inputs(*shape, BF16, seed=12)
    w = dict(causal=True, window=window, sinks=sinks)
    o, lse = R.forward(q, k, v, **w)
    got = ta.attention_backward(d_o, q, k, v, o.to(BF16), lse.float(), **w)
    R.check(got, *R.backward(d_o, q, k, v, **w))
    again = ta.attention_backward(d_o, q, k, v, o.to(BF16), lse.float(), **w)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("masked", [False, True])
def test_fp16_keeps_its_bits_over_many_keys(masked):
    """P of 1/6000 and dS of a few 1e-5 lie below fp16's normal numbers. A rounding is off by 2^-11 / sqrt(3) of the value (in the
    mean square, at the worst mantissa); an operand's and the result's are independent, so that thousands of them together
    are off by sqrt(2) of that."""
    d_o, q, k, v = _inputs(1, 1, 1, 6000, 6000, 128, F16, seed=13)
    d_o.mul_(0.01)
    kw = dict(mask=torch.zeros((1, 6000, 6000), device="cuda")) if masked else {}
    got = _run(d_o, q, k, v, **kw)
    want, _ = R.backward(d_o, q, k, v, **kw)
    for name, a, w in zip(("dq", "dk", "dv"), got, want):
        assert float((a.double() - w).norm() / w.norm()) < 2 ** -11 * (2 / 3) ** 0.5, name


@pytest.mark.gpu
@pytest.mark.parametrize("factor", [0.0, 2.0 ** -14, 1.0, 4000.0])
def test_fp16_over_its_range(factor):
    """dO from nothing to where a key alone in its row would leave fp16, among rows that see one key or two."""
    d_o, q, k, v = _inputs(1, 4, 2, 200, 200, 64, F16, seed=14)
    d_o.mul_(factor)
    _check(d_o, q, k, v, causal=True, label=str(factor))


def _mask(kind, B, Sq, Sk, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(5)
    m = torch.zeros((B, Sq, Sk), device=dev)
    if kind == "holes":
        m.masked_fill_(torch.rand((B, Sq, Sk), device=dev, generator=g) < 0.3, float("-inf"))
        m[:, 3::17] = float("-inf")
    elif kind == "bias":
        m.normal_(generator=g).mul_(3)
    elif kind == "lowest":                       # padding by the type's lowest value; some rows hold nothing else
        m[:, :, Sk // 2:] = torch.finfo(torch.float32).min
    elif kind == "large":                        # rows whose every key is pushed away by the same large value
        m[:, 2::5] = -1e4
        m[:, 1::3, : Sk // 3] = -1e9
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("kind", ["holes", "bias", "lowest", "large"])
@pytest.mark.parametrize("shape,dtype", [((2, 2, 1, 200, 300, 64), BF16), ((1, 2, 2, 131, 259, 128), F16),
                                         ((1, 2, 2, 384, 256, 128), BF16)])
def test_additive_masks(shape, dtype, kind, causal):
    mask = _mask(kind, shape[0], shape[3], shape[4])
    _check(*_inputs(*shape, dtype, seed=4), mask=mask, causal=causal, label=kind)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [-1e9, -1e30, torch.finfo(torch.float32).min, float("-inf")])
def test_rows_pushed_away_whole(value):
    """Rows of padding: their own gradients are finite, and with dO = 0 there they leave no trace in dK and dV."""
    d_o, q, k, v = _inputs(1, 2, 1, 200, 200, 64, BF16, seed=6)
    d_o[:, 150:] = 0
    mask = torch.zeros((1, 200, 200), device="cuda")
    mask[:, 150:] = value
    o, lse = ta.attention(q, k, v, mask=mask)
    dq, dk, dv = ta.attention_backward(d_o, q, k, v, o, lse, mask=mask)
    assert bool((dq[:, 150:] == 0).all())
    want, bounds = R.backward(d_o[:, :150], q[:, :150], k, v)
    R.check((dq[:, :150], dk, dv), want, [2 * b for b in bounds])      # (o and lse of the forward call: see below)


@pytest.mark.gpu
def test_rows_pushed_away_share_their_weight():
    """A row whose every logit is the same large number (the mask takes the logits' bits) has uniform probabilities."""
    d_o, q, k, v = _inputs(1, 1, 1, 130, 256, 64, BF16, seed=7)
    mask = torch.full((1, 130, 256), -2.0 ** 40, device="cuda")
    o, lse = ta.attention(q, k, v, mask=mask)
    _, _, dv = ta.attention_backward(d_o, q, k, v, o, lse, mask=mask)
    want = d_o.double().sum(1, keepdim=True) / 256                    # (weights of 1 / 256: exact in bf16)
    assert bool(((dv.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * d_o.double().abs().sum(1)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
def test_through_the_forward_call_and_a_packed_projection(D, dtype):
    """What a training step does: the forward call's own o and lse, Q, K, V and their gradients inside packed tensors."""
    B, S, Hq, Hkv = 2, 333, 6, 2
    F = (Hq + 2 * Hkv) * D
    g = torch.Generator(device="cuda").manual_seed(8)
    qkv = torch.empty((B, S, F), dtype=dtype, device="cuda").normal_(generator=g)
    d_o = torch.empty((B, S, Hq, D), dtype=dtype, device="cuda").normal_(generator=g)
    parts = (Hq * D, Hkv * D, Hkv * D)
    q, k, v = (t.unflatten(-1, (t.shape[-1] // D, D)) for t in qkv.split(parts, dim=-1))
    o, lse = ta.attention(q.contiguous(), k.contiguous(), v.contiguous(), causal=True)
    d_qkv = torch.full_like(qkv, float("nan"))
    grads = [t.unflatten(-1, (t.shape[-1] // D, D)) for t in d_qkv.split(parts, dim=-1)]
    got = ta.attention_backward(d_o, q, k, v, o, lse, causal=True, dq=grads[0], dk=grads[1], dv=grads[2])
    assert all(a is b for a, b in zip(got, grads))
    want, bounds = R.backward(d_o, q, k, v, causal=True)
    # the forward call's o is off by P's rounding too (half a step of each weight): delta by that much again, and lse by
    # FP32 steps; twice the bound holds both
    R.check(got, want, [2 * b for b in bounds])
    plain = ta.attention_backward(d_o, q.contiguous(), k.contiguous(), v.contiguous(), o, lse, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(got, plain))


@pytest.mark.gpu
def test_odd_strides_and_offsets():
    """Tokens 8 elements further apart than they need be, starting 16 bytes into their storage."""
    B, S, H, D = 2, 200, 2, 64
    def odd(seed):
        base = torch.empty(8 + B * S * (H * D + 8), dtype=BF16, device="cuda")
        t = base[8:].view(B, S, H * D + 8)[:, :, :H * D].unflatten(-1, (H, D))
        return t.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
    q, k, v = odd(1), odd(2), odd(3)
    d_o = q.contiguous().roll(1, 0)
    o, lse = R.forward(q, k, v, causal=True)
    o, lse = o.to(BF16), lse.float()
    dq, dk, dv = odd(4), odd(5), odd(6)
    got = ta.attention_backward(d_o, q, k, v, o, lse, causal=True, dq=dq, dk=dk, dv=dv)
    R.check(got, *R.backward(d_o, q, k, v, causal=True))


@pytest.mark.gpu
def test_empty_sizes_give_zero_gradients():
    for Sq, Sk in ((0, 5), (5, 0), (0, 0)):
        d_o, q, k, v = _inputs(2, 4, 2, Sq, Sk, 64, BF16)
        o, lse = torch.zeros_like(q), torch.full((2, 4, Sq), float("-inf"), device="cuda")
        grads = [torch.full_like(t, float("nan")) for t in (q, k, v)]
        ta.attention_backward(d_o, q, k, v, o, lse, dq=grads[0], dk=grads[1], dv=grads[2])
        assert all(bool((t == 0).all()) for t in grads)
    # queries before the first key and keys behind the last query of a window see nothing
    _check(*_inputs(1, 1, 1, 400, 30, 64, BF16), causal=True)
    _check(*_inputs(1, 1, 1, 20, 900, 64, BF16), causal=True, window=10)


@pytest.mark.gpu
@pytest.mark.parametrize("masked", [False, True])
def test_many_tiles_without_a_pair(masked):
    """Several in a row for every CTA: queries before all keys, keys that no window reaches."""
    mask = _mask("bias", 4, 1000, 100) if masked else None
    _check(*_inputs(4, 32, 16, 1000, 100, 64, BF16, seed=15), causal=True, mask=mask)
    if not masked:
        _check(*_inputs(4, 32, 32, 50, 2000, 128, BF16, seed=16), causal=True, window=20)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.02, 1.0, 3.0])
def test_scales(scale):
    _check(*_inputs(1, 2, 1, 200, 200, 128, BF16, seed=9), causal=True, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-4, 1.0, 3e3])
def test_small_and_large_gradients_in_fp16(size):
    _check(*_inputs(1, 2, 1, 500, 500, 64, F16, seed=10, size=size), causal=True)


@pytest.mark.gpu
def test_the_same_from_run_to_run_and_on_another_stream():
    d_o, q, k, v = _inputs(2, 8, 2, 600, 600, 128, BF16, seed=11)
    o, lse = ta.attention(q, k, v, causal=True)
    first = ta.attention_backward(d_o, q, k, v, o, lse, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = ta.attention_backward(d_o, q, k, v, o, lse, causal=True, stream=side)
    with torch.cuda.stream(side):
        b = ta.attention_backward(d_o, q, k, v, o, lse, causal=True)
    torch.cuda.synchronize()
    for other in (a, b, ta.attention_backward(d_o, q, k, v, o, lse, causal=True)):
        assert all(torch.equal(x, y) for x, y in zip(first, other))


@pytest.mark.gpu
def test_two_captured_steps_replayed():
    """A forward and backward step captured twice, each with its own workspace, replayed with new inputs."""
    d_o, q, k, v = _inputs(1, 4, 2, 300, 300, 64, BF16, seed=12)

    def step():
        o, lse = ta.attention(q, k, v, causal=True)
        return ta.attention_backward(d_o, q, k, v, o, lse, causal=True)

    step()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(step())
            graphs.append(g)
    new = _inputs(1, 4, 2, 300, 300, 64, BF16, seed=13)
    for t, n in zip((d_o, q, k, v), new):
        t.copy_(n)
    torch.cuda.synchronize()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = step()
    for out in outs:
        assert all(torch.equal(x, y) for x, y in zip(out, want))


@pytest.mark.gpu
def test_long_sequences_past_32_bit_offsets():
    """dQ and dK of a tensor whose last rows lie past 2^31 elements, compared on the last head alone."""
    B, S, H, D = 1, 140000, 120, 128                                   # 2.15e9 elements, 4.3 GB a tensor
    d_o, q, k, v = _inputs(B, H, H, S, S, D, BF16, seed=14)
    o, lse = ta.attention_window(q, k, v, window=64)
    dq, dk, dv = ta.attention_backward(d_o, q, k, v, o, lse, causal=True, window=64)
    tail = slice(S - 512, S)
    part = [t[:, tail, H - 1:].contiguous() for t in (d_o, q, k, v)]
    want, bounds = R.backward(*part, causal=True, window=64)
    got = [t[:, tail, H - 1:] for t in (dq, dk, dv)]
    # queries whose window lies whole in the part; their keys' queries do as well
    R.check([t[:, 64:] for t in got], [t[:, 64:] for t in want], [2 * t[:, 64:] for t in bounds])


@pytest.mark.gpu
def test_refusals_of_tensors():
    d_o, q, k, v = _inputs(1, 4, 2, 64, 64, 64, BF16)
    o, lse = ta.attention(q, k, v)
    ok = dict(d_o=d_o, q=q, k=k, v=v, o=o, lse=lse)

    def call(**kw):
        a = dict(ok, **kw)
        return ta.attention_backward(a.pop("d_o"), a.pop("q"), a.pop("k"), a.pop("v"), a.pop("o"), a.pop("lse"), **a)

    call()
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(q=q.cpu()), dict(v=v[:, :5]), dict(o=o[:, :5]), dict(lse=lse.half()),
                dict(d_o=d_o.transpose(1, 2)), dict(lse=lse[..., :5]), dict(q=q.transpose(1, 2)), dict(dq=k.clone()),
                dict(window=5), dict(window=-1, causal=True), dict(window=5, causal=True, mask=torch.zeros(1, 64, 64).cuda()),
                dict(mask=torch.zeros(64, 64).cuda()), dict(mask=torch.zeros(1, 64, 64)), dict(workspace=torch.empty(8)),
                dict(o=o[0]), dict(dk=torch.empty_like(k, dtype=F16))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ta.AttnError):
        call(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ta.AttnError):
        call(q=q[..., :32].contiguous(), k=k[..., :32].contiguous(), v=v[..., :32].contiguous(), o=o[..., :32].contiguous(),
             d_o=d_o[..., :32].contiguous())


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported():
    d_o, q, k, v = _inputs(1, 2, 2, 300, 300, 64, BF16)
    o, lse = ta.attention(q, k, v)
    stream = torch.cuda.current_stream().cuda_stream
    try:
        A.attn_set_wait_timeout_ns(20_000_000)
        A.attn_debug_inject_stall(True)
        ta.attention_backward(d_o, q, k, v, o, lse)
        assert A.attn_last_status(stream) == A.ATTN_ERR_DEVICE_TIMEOUT
    finally:
        A.attn_debug_inject_stall(False)
        A.attn_set_wait_timeout_ns(0)
    _check(d_o, q, k, v)


# ----------------------------------------------------- host checks, no GPU

P = 0x10000


def _raw(fn=A.attn_bwd, g=2 * P, q=3 * P, k=4 * P, v=5 * P, o=6 * P, lse=7 * P, dq=8 * P, dk=9 * P, dv=10 * P, st=None, B=1, Hq=2,
         Hkv=2, Sq=16, Sk=16, D=64, kind=0, mask=None, window=0, sinks=0, ws=P, ws_bytes=1 << 20):
    st = st or [Hq * D, Hkv * D, Hkv * D] * 2
    return fn(g, q, k, v, o, lse, dq, dk, dv, *st, B, Hq, Hkv, Sq, Sk, D, 0.0, kind, mask, window, sinks, ws, ws_bytes, None)


@pytest.mark.parametrize("fn", [A.attn_bwd, A.attn_bwd_f16])
@pytest.mark.parametrize("kw,code", [
    *[({n: None}, 1) for n in ("g", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "ws")],
    *[({n: P + 8}, 1) for n in ("g", "q", "k", "v", "o", "dq", "dk", "dv", "ws")],
    (dict(lse=P + 2), 1), (dict(B=-1), 1), (dict(Sq=-1), 1), (dict(Sk=-1), 1), (dict(Hkv=0), 1), (dict(Hq=3), 1),
    (dict(kind=4), 1), (dict(kind=-1), 1), (dict(kind=2), 1), (dict(kind=2, mask=P + 1), 1), (dict(window=-1), 1),
    (dict(kind=1, sinks=-1), 1), (dict(kind=0, window=3), 1), (dict(kind=3, mask=P, window=3), 1), (dict(ws_bytes=100), 1),
    (dict(st=[120, 128, 128, 128, 128, 128]), 1), (dict(st=[132, 128, 128, 128, 128, 128]), 1),
    (dict(st=[128, 128, 128, 128, 128, 64]), 1), (dict(D=96), 2), (dict(Sq=(1 << 30) + 1), 1),
    *[({out: n * P}, 1) for out in ("dq", "dk", "dv") for n in range(1, 11) if n != 8 + ("dq", "dk", "dv").index(out)],
    (dict(kind=2, mask=9 * P), 1),
    (dict(B=0), 0), (dict(Sq=0, Sk=0), 0), (dict(B=1 << 20, Sq=1 << 20, Sk=1 << 20), 1),
])
def test_refusals_on_the_host(fn, kw, code):
    assert _raw(fn, **kw) == code


def test_workspace_sizes():
    # (8 and 12 tiles of dQ and of dK, dV, too short to be cut)
    assert A.attn_bwd_workspace_bytes(2, 4, 2, 100, 300, 64, 1) == 1024 + 2 * 2 * 4 * 128 * 4
    assert A.attn_bwd_workspace_bytes(2, 4, 2, 100, 300, 64, 2) == 1024 + 3 * 2 * 4 * 128 * 4
    # one tile of 64 blocks of 128 keys: 16 parts of dQ of 1 x 128 x 64 FP32 values; the longer walk of dK and dV has one block
    assert A.attn_bwd_workspace_bytes(1, 1, 1, 128, 8192, 64, 1) == 1024 + 2 * 128 * 4 + 16 * 128 * 64 * 4
    assert A.attn_bwd_workspace_bytes(2, 4, 3, 100, 300, 64, 1) == 0
    assert A.attn_bwd_workspace_bytes(2, 4, 2, 0, 300, 64, 1) == 0
