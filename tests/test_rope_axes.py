"""Rotary positions with several axes against complex multiplication in 64 bits by the table's own entries."""
import ctypes

import pytest
import torch

import transformer_attention_02_gb300 as ta
from transformer_attention_02_gb300 import attn as A

BF16, F16 = torch.bfloat16, torch.float16


def _table(max_pos, D, dev="cuda"):
    theta = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)
    return torch.stack([theta.cos(), theta.sin()], -1).float().to(dev)


def _want(x, table, positions, sections, inverse):
    """(values, bounds): half a step of the type for the one rounding, two FP32 steps of each product."""
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(x.device)
    a = table.double()[positions.long()[..., axis], torch.arange(sum(sections), device=x.device)][:, :, None]
    c, s = a[..., 0], -a[..., 1] if inverse else a[..., 1]
    x0, x1 = x[..., 0::2].double(), x[..., 1::2].double()
    y = torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], -1).flatten(-2)
    size = torch.stack([(x0 * c).abs() + (x1 * s).abs(), (x1 * c).abs() + (x0 * s).abs()], -1).flatten(-2)
    tiny = 2.0 ** -25 if x.dtype == F16 else 2.0 ** -126
    return y, torch.finfo(x.dtype).eps / 2 * y.abs() + 2.0 ** -22 * size + tiny


def _check(got, x, *args):
    y, bound = _want(x, *args)
    assert bool(((got.double() - y).abs() <= bound).all())


def _inputs(B, S, Hq, Hkv, D, dtype, axes, max_pos, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.empty((B, S, Hq, D), dtype=dtype, device="cuda").normal_(generator=g)
    k = torch.empty((B, S, Hkv, D), dtype=dtype, device="cuda").normal_(generator=g)
    pos = torch.randint(0, max_pos, (B, S, axes), device="cuda", generator=g, dtype=torch.int32)
    return q, k, pos


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,S,Hq,Hkv,sections", [
    (1, 1, 1, 1, (32,)),
    (32, 1, 32, 8, (16, 24, 24)),
    (2, 300, 8, 2, (16, 24, 24)),
    (3, 77, 5, 5, (8, 12, 12)),
    (2, 130, 3, 1, (1, 2, 29)),              # sections that end inside a 16-byte piece
    (2, 65, 4, 2, (0, 31, 0, 33)),           # axes without pairs
    (1, 700, 2, 2, (7, 41)),                 # 96 values: pieces that do not divide 32
    (1, 9, 3, 1, (4,)),
    (1, 5, 2, 1, (100, 156, 256)),           # a head vector of 1024
    (1, 4000, 40, 8, (32, 16, 16)),
])
def test_values(B, S, Hq, Hkv, sections, dtype, inverse):
    D = 2 * sum(sections)
    q, k, pos = _inputs(B, S, Hq, Hkv, D, dtype, len(sections), 5000)
    table = _table(5000, D)
    q2, k2 = ta.rope_axes(q, k, table, pos, sections, inverse=inverse)
    _check(q2, q, table, pos, sections, inverse)
    _check(k2, k, table, pos, sections, inverse)
    alone = ta.rope_axes(q, None, table, pos, sections, inverse=inverse)
    assert torch.equal(alone, q2)
    ta.rope_axes(q, k, table, pos, sections, inverse=inverse, q_out=q, k_out=k)              # in place
    assert torch.equal(q, q2) and torch.equal(k, k2)


@pytest.mark.gpu
def test_one_axis_is_rope_apply_and_the_way_back_returns():
    q, k, _ = _inputs(2, 200, 4, 2, 128, BF16, 1, 10)
    table = ta.rope_table(300, 128)
    pos = (torch.arange(200, device="cuda", dtype=torch.int32) + 50).expand(2, 200)[..., None].contiguous()
    q2, k2 = ta.rope_axes(q, k, table, pos, [64])
    assert torch.equal(q2, ta.rope_apply(q, table, pos0=50)) and torch.equal(k2, ta.rope_apply(k, table, pos0=50))
    back = ta.rope_axes(q2, None, table, pos, [64], inverse=True)
    # two roundings, each of half a step of a vector pair's length, which a rotation keeps
    size = q.double().unflatten(-1, (64, 2)).norm(dim=-1, keepdim=True).expand(-1, -1, -1, -1, 2).flatten(-2)
    assert bool(((back.double() - q.double()).abs() <= 3 * 2.0 ** -8 * size).all())


@pytest.mark.gpu
def test_the_gradient_is_the_transpose():
    """<rot(x), y> = <x, rot^-1(y)>, up to the roundings of both sides (half a step of each value)."""
    x, y, pos = _inputs(2, 50, 6, 6, 64, BF16, 3, 4000)
    table = ta.rope_axes_table(4000, (8, 12, 12))
    a = ta.rope_axes(x, None, table, pos, (8, 12, 12)).double()
    b = ta.rope_axes(y, None, table, pos, (8, 12, 12), inverse=True).double()
    left, right = (a * y.double()).sum(), (x.double() * b).sum()
    slack = 2.0 ** -8 * ((a * y.double()).abs().sum() + (x.double() * b).abs().sum())
    assert abs(float(left - right)) <= float(slack)


@pytest.mark.gpu
@pytest.mark.parametrize("sections", [(16, 24, 24), (8, 12, 12), (5,), (0, 7)])
def test_table_of_own_frequencies(sections):
    """Angles up to pos: FP64 on both sides, so the FP32 entries differ by half a step of 1 and the angles' own rounding."""
    table = ta.rope_axes_table(3000, sections, 500.0)
    e = torch.cat([torch.arange(n, dtype=torch.float64) / max(n, 1) for n in sections])
    theta = torch.arange(3000, dtype=torch.float64)[:, None] * 500.0 ** -e
    want = torch.stack([theta.cos(), theta.sin()], -1).to("cuda")
    assert table.shape == (3000, sum(sections), 2)
    assert float((table.double() - want).abs().max()) <= 2.0 ** -25 + 3000 * 2.0 ** -50


@pytest.mark.gpu
def test_slices_of_a_packed_projection():
    B, S, Hq, Hkv, D = 2, 123, 6, 2, 128
    F = (Hq + 2 * Hkv) * D
    qkv = torch.empty((B, S, F), dtype=BF16, device="cuda").normal_()
    before = qkv.clone()
    q, k, v = (t.unflatten(-1, (t.shape[-1] // D, D)) for t in qkv.split((Hq * D, Hkv * D, Hkv * D), dim=-1))
    _, _, pos = _inputs(B, S, 1, 1, D, BF16, 3, 900)
    table = _table(900, D)
    want = ta.rope_axes(q.contiguous(), k.contiguous(), table, pos, (16, 24, 24))
    ta.rope_axes(q, k, table, pos, (16, 24, 24), q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[..., (Hq + Hkv) * D:], before[..., (Hq + Hkv) * D:])


@pytest.mark.gpu
def test_positions_out_of_range_leave_their_tokens():
    q, k, pos = _inputs(2, 40, 3, 1, 64, F16, 2, 100)
    pos[0, 3, 1], pos[1, 39, 0], pos[1, 7, 0] = 100, -1, 2 ** 31 - 1
    table = _table(100, 64)
    q2, k2 = torch.full_like(q, 7), torch.full_like(k, 7)
    stream = torch.cuda.current_stream().cuda_stream
    ta.rope_axes(q, k, table, pos, (10, 22), q_out=q2, k_out=k2)
    assert A.attn_last_status(stream) == A.ATTN_ERR_BAD_INDEX
    assert A.attn_last_status(stream) == A.ATTN_OK
    bad = torch.zeros((2, 40), dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[1, 39] = bad[1, 7] = True
    assert bool((q2[bad] == 7).all()) and bool((k2[bad] == 7).all())
    y, bound = _want(q, table, pos.clamp(0, 99), (10, 22), False)
    assert bool(((q2.double() - y).abs() <= bound)[~bad].all())


@pytest.mark.gpu
def test_nothing_to_turn_and_other_streams():
    table = _table(64, 64)
    q, k, pos = _inputs(2, 0, 3, 1, 64, BF16, 1, 10)
    assert ta.rope_axes(q, k, table, pos, [32])[0].shape == (2, 0, 3, 64)
    q, k, pos = _inputs(2, 33, 3, 1, 64, BF16, 2, 64)
    want = ta.rope_axes(q, k, table, pos, [8, 24])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ta.rope_axes(q, k, table, pos, [8, 24], stream=side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = ta.rope_axes(q, k, table, pos, [8, 24])
    pos.copy_(pos.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(captured, ta.rope_axes(q, k, table, pos, [8, 24])))


@pytest.mark.gpu
def test_refusals_of_tensors():
    q, k, pos = _inputs(2, 30, 4, 2, 64, BF16, 2, 50)
    table = _table(50, 64)
    ok = dict(q=q, k=k, table=table, positions=pos, sections=(8, 24))
    ta.rope_axes(**ok)
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(k=k[:, :5]), dict(positions=pos.long()), dict(positions=pos[..., :1]),
                dict(positions=pos.cpu()), dict(sections=(8, 23)), dict(sections=(8, 8, 16)), dict(sections=()),
                dict(sections=(-8, 40)), dict(table=table[:, :16]), dict(table=table.double()), dict(table=table[:0]),
                dict(q=q.transpose(1, 2)), dict(q_out=k), dict(k=None, k_out=k), dict(k_out=k.half()), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            ta.rope_axes(**dict(ok, **bad))


# ----------------------------------------------------- host checks, no GPU

P = 0x10000


def _raw(fn=A.attn_rope_axes, q=P, qo=2 * P, qs=256, qos=256, k=3 * P, ko=4 * P, ks=128, kos=128, B=1, S=4, Hq=4, Hkv=2, D=64,
         table=5 * P, max_pos=16, pos=6 * P, sections=(8, 24), n=None, inverse=0):
    s = None if sections is None else (ctypes.c_int * max(1, len(sections)))(*sections)
    return fn(q, qo, qs, qos, k, ko, ks, kos, B, S, Hq, Hkv, D, table, max_pos, pos, s,
              len(sections or ()) if n is None else n, inverse, None)


@pytest.mark.parametrize("fn", [A.attn_rope_axes, A.attn_rope_axes_f16])
@pytest.mark.parametrize("kw,code", [
    *[({n: None}, 1) for n in ("q", "qo", "k", "ko", "table", "pos", "sections")],
    *[({n: P + 8}, 1) for n in ("q", "qo", "k", "ko")], (dict(table=P + 4), 1), (dict(pos=P + 2), 1),
    (dict(qs=255), 1), (dict(qs=260), 1), (dict(kos=120), 1), (dict(B=-1), 1), (dict(S=-1), 1), (dict(Hq=-1), 1), (dict(D=60), 1),
    (dict(D=0), 1), (dict(D=2048), 1), (dict(max_pos=0), 1), (dict(sections=(8, 23)), 1), (dict(sections=(8, 25)), 1),
    (dict(qo=3 * P), 1), (dict(ko=P), 1), (dict(ko=2 * P), 1), (dict(qo=P, qos=264), 1), (dict(ko=3 * P, kos=136), 1),
    (dict(sections=(-1, 33)), 1), (dict(n=0), 1), (dict(sections=(8, 8, 8, 4, 4)), 1), (dict(B=0), 0), (dict(S=0), 0),
    (dict(Hq=0, Hkv=0), 0),
])
def test_refusals_on_the_host(fn, kw, code):
    assert _raw(fn, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), 1), (dict(max_pos=-1), 1), (dict(max_pos=0), 0), (dict(sections=(0, 0)), 1), (dict(sections=(-1, 5)), 1),
    (dict(sections=(600,)), 1), (dict(base=1.0), 1), (dict(base=float("nan")), 1), (dict(max_pos=2 ** 30, sections=(8,)), 1),
])
def test_table_refusals_on_the_host(kw, code):
    a = dict(dict(table=P, max_pos=10, sections=(8, 24), base=10000.0), **kw)
    s = (ctypes.c_int * len(a["sections"]))(*a["sections"])
    assert A.attn_rope_axes_table(a["table"], a["max_pos"], s, len(a["sections"]), a["base"], None) == code
