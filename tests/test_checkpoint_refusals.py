"""What the checkpoints' entry points refuse, each argument at an address of its own, so that a refusal can only be of what a case
changes. Only where there is no GPU, since the addresses are no memory."""
import pytest
import torch

from transformer_attention_02_gb300 import attn as A

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="calls with addresses that are no memory")

P = 0x10000
INVALID = 1


def _store(fn, **kw):
    a = dict(dict(x=P, stride=128, codes=2 * P, scale=3 * P, B=1, S=4, H=2, D=64), **kw)
    if fn in (A.attn_checkpoint_store, A.attn_checkpoint_store_f16):
        return fn(a["x"], a["stride"], a["codes"], a["scale"], a["B"], a["S"], a["H"], a["D"], None)
    return fn(a["codes"], a["scale"], a["x"], a["stride"], a["B"], a["S"], a["H"], a["D"], None)


BACK = dict(g=P, q=2 * P, k=3 * P, v=4 * P, qs=5 * P, ks=6 * P, vs=7 * P, dq=8 * P, dk=9 * P, dv=10 * P, st=[128, 128, 128], B=1, Hq=2,
            Hkv=2, Sq=16, Sk=16, D=64, kind=0, mask=None, window=0, sinks=0, ws=12 * P, size=1 << 20)


def _backward(fn, **kw):
    a = dict(BACK, **kw)
    return fn(a["g"], a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["dq"], a["dk"], a["dv"], *a["st"], a["B"], a["Hq"], a["Hkv"],
              a["Sq"], a["Sk"], a["D"], 0.0, a["kind"], a["mask"], a["window"], a["sinks"], a["ws"], a["size"], None)


CONVERSIONS = [A.attn_checkpoint_store, A.attn_checkpoint_store_f16, A.attn_checkpoint_load, A.attn_checkpoint_load_f16]
BACKWARDS = [A.attn_bwd_checkpoint, A.attn_bwd_checkpoint_f16]


@pytest.mark.parametrize("fn", CONVERSIONS)
@pytest.mark.parametrize("kw", [dict(codes=P), dict(scale=P), dict(scale=2 * P)])
def test_a_conversion_onto_itself_is_refused(fn, kw):
    assert _store(fn) != INVALID
    assert _store(fn, **kw) == INVALID


@pytest.mark.parametrize("fn", BACKWARDS)
@pytest.mark.parametrize("out", ["dq", "dk", "dv", "ws"])
@pytest.mark.parametrize("at", ["g", "q", "k", "v", "qs", "ks", "vs", "dq", "dk", "dv", "ws"])
def test_gradients_onto_other_tensors_are_refused(fn, out, at):
    assert _backward(fn) != INVALID
    if at != out:
        assert _backward(fn, **{out: BACK[at]}) == INVALID


@pytest.mark.parametrize("fn", CONVERSIONS)
@pytest.mark.parametrize("kw,code", [
    *[({n: None}, 1) for n in ("x", "codes", "scale")], *[({n: 15 * P + 8}, 1) for n in ("x", "codes")], (dict(scale=15 * P + 2), 1),
    (dict(stride=120), 1), (dict(stride=132), 1), (dict(B=-1), 1), (dict(S=-1), 1), (dict(H=-1), 1), (dict(D=96), 2), (dict(D=0), 1),
    (dict(B=1 << 30, S=1 << 30), 1), (dict(B=0), 0), (dict(S=0), 0), (dict(H=0), 0),
])
def test_conversions(fn, kw, code):
    assert _store(fn) != INVALID
    assert _store(fn, **kw) == code


@pytest.mark.parametrize("fn", BACKWARDS)
@pytest.mark.parametrize("kw,code", [
    *[({n: None}, 1) for n in ("g", "q", "k", "v", "qs", "ks", "vs", "dq", "dk", "dv", "ws")],
    *[({n: 15 * P + 8}, 1) for n in ("g", "q", "k", "v", "dq", "dk", "dv", "ws")],
    *[({n: 15 * P + 1}, 1) for n in ("qs", "ks", "vs")], (dict(ws=15 * P + 128), 1),
    *[(dict(st=[s if i == n else 128 for i in range(3)]), 1) for n in range(3) for s in (120, 132, 64)],
    (dict(kind=-1), 1), (dict(kind=4), 1), (dict(kind=5), 1), (dict(window=2), 1), (dict(kind=1, window=-1), 1), (dict(kind=1, sinks=-1), 1),
    (dict(kind=3, mask=14 * P, window=2), 1), (dict(kind=2), 1), (dict(kind=3), 1), (dict(kind=2, mask=14 * P + 1), 1),
    (dict(size=1000), 1), (dict(B=-1), 1), (dict(Sq=-1), 1), (dict(Sk=-1), 1), (dict(Hkv=0), 1), (dict(Hq=3), 1), (dict(Sq=(1 << 30) + 1), 1),
    (dict(D=32), 2), (dict(D=96), 2), (dict(B=0), 0), (dict(Sq=0, Sk=0), 0),
])
def test_backward(fn, kw, code):
    assert _backward(fn) != INVALID
    assert _backward(fn, **kw) == code


@pytest.mark.parametrize("fn", BACKWARDS)
@pytest.mark.parametrize("kw", [dict(kind=1), dict(kind=1, window=5, sinks=2), dict(kind=2, mask=14 * P), dict(kind=3, mask=14 * P),
                                dict(D=128, st=[256, 256, 264]), dict(Hq=4, st=[256, 128, 128])])
def test_other_calls_that_are_none_of_these(fn, kw):
    assert _backward(fn, **kw) != INVALID


@pytest.mark.parametrize("fn", BACKWARDS)
def test_the_workspace_is_as_large_as_the_call_says(fn):
    size = A.attn_bwd_checkpoint_workspace_bytes(1, 2, 2, 16, 16, 64, 0)
    assert _backward(fn, size=size) != INVALID and _backward(fn, size=size - 1) == INVALID
