"""Causal attention with a sliding window and sinks (attn_fwd_window) against the plain 64-bit form of paged_ref (the
bounds are derived there), and its relations to the causal kernel."""
import numpy as np
import pytest
import torch

import paged_ref as R
from transformer_attention_02_gb300 import attn as A

BF, FP = torch.bfloat16, torch.float16
P = 0x10000


def _qkv(B, Hq, Hkv, Sq, Sk, D, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(dt).cuda() for s in ((B, Sq, Hq, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D))]


CASES = [
    # B, Hq, Hkv, Sq, Sk, D, window, sinks
    (1, 2, 2, 1, 1, 64, 1, 0),
    (1, 2, 1, 300, 300, 128, 1, 0),            # each query sees itself alone
    (2, 2, 2, 300, 300, 64, 40, 3),
    (1, 4, 2, 700, 700, 128, 128, 0),          # windows that begin at block edges
    (1, 4, 1, 900, 900, 128, 130, 4),          # a gap between the sinks' block and the window
    (1, 2, 2, 900, 900, 64, 200, 140),         # sinks over two blocks
    (1, 2, 2, 100, 1000, 128, 300, 7),         # Sq < Sk
    (1, 2, 2, 400, 150, 64, 50, 2),            # Sq > Sk: leading rows see no key
    (1, 2, 2, 1, 777, 128, 100, 5),            # one token
    (1, 6, 2, 513, 513, 64, 512, 1),
    (1, 2, 1, 640, 640, 128, 639, 0),          # one key short of hiding nothing
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "f16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}_H{}-{}_S{}-{}_D{}_w{}s{}".format(*c))
def test_window_matches_plain_form(case, dt):
    B, Hq, Hkv, Sq, Sk, D, window, sinks = case
    q, k, v = _qkv(B, Hq, Hkv, Sq, Sk, D, dt, sum(case))
    o, lse = A.attention_window(q, k, v, window=window, sinks=sinks)
    assert A.attn_last_status(torch.cuda.current_stream().cuda_stream) == A.ATTN_OK
    for b in range(B):
        want = R.attend(R.f64(q[b]), R.f64(k[b]), R.f64(v[b]), np.arange(Sq) + Sk - Sq, D ** -0.5, window, sinks)
        R.check_rows(R.f64(o[b]), R.f64(lse[b]), want, R.step(dt), R.step(dt), D, Sk, float(v[b].float().abs().max()),
                     str(case))
    o2, lse2 = A.attention_window(q, k, v, window=window, sinks=sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(500, 0), (1 << 30, 0), (3, 500), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_a_window_that_hides_nothing_is_the_causal_kernel(window, sinks):
    q, k, v = _qkv(1, 4, 2, 500, 500, 128, BF, 1)
    o, lse = A.attention_window(q, k, v, window=window, sinks=sinks)
    o2, lse2 = A.attention(q, k, v, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_blocks_outside_the_window_are_not_read():
    """NaN in every key block that no row of the last tile sees leaves that tile's rows as they were."""
    q, k, v = _qkv(1, 2, 2, 2048, 2048, 128, BF, 2)
    clean = A.attention_window(q, k, v, window=256, sinks=4)
    for t in (k, v):
        t[:, 128:1536] = float("nan")                  # the last tile's rows 1792..2047 see 1537.. and 0..3
    o, lse = A.attention_window(q, k, v, window=256, sinks=4)
    assert torch.equal(o[:, 1792:], clean[0][:, 1792:]) and torch.equal(lse[..., 1792:], clean[1][..., 1792:])


@pytest.mark.gpu
def test_long_window_against_the_masked_kernel():
    """The benchmark's GQA prefill heads at 4096 keys: the same visibility as an additive mask of the existing kernel."""
    q, k, v = _qkv(1, 8, 2, 4096, 4096, 128, BF, 3)
    o, lse = A.attention_window(q, k, v, window=1000, sinks=4)
    i, j = torch.arange(4096, device="cuda")[:, None], torch.arange(4096, device="cuda")[None]
    mask = torch.where((j > i - 1000) | (j < 4), 0.0, float("-inf")).float()[None].contiguous()
    o2, lse2 = A.attention(q, k, v, causal=True, mask=mask)
    # both round the same weights to bf16 under maxima up to 2^8 apart, a step 2^-8 each of sum p|v| <= max|v|
    assert float((o.float() - o2.float()).abs().max()) <= 2 * 2.0 ** -8 * (float(v.float().abs().max()) + 1)
    assert float((lse - lse2).abs().max()) <= 1e-4


@pytest.mark.gpu
def test_window_in_a_graph_and_on_a_side_stream():
    q, k, v = _qkv(1, 4, 4, 600, 600, 64, FP, 4)
    want = A.attention_window(q, k, v, window=77, sinks=1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, lse = A.attention_window(q, k, v, window=77, sinks=1, stream=s)
    assert A.attn_last_status(s.cuda_stream) == A.ATTN_OK
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    out, l2 = torch.empty_like(q), torch.empty_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.attention_window(q, k, v, window=77, sinks=1, out=out, lse=l2)
    q.copy_(torch.roll(q, 1, 1))
    g.replay()
    torch.cuda.synchronize()
    want = A.attention_window(q, k, v, window=77, sinks=1)
    assert torch.equal(out, want[0]) and torch.equal(l2, want[1])


@pytest.mark.gpu
def test_windowed_prompt_then_windowed_decode():
    """A windowed prompt and single tokens over a 16-bit cache: each token's attention over the cache equals the last row
    of attention_window over everything so far, up to the rounding of the weights."""
    B, Hq, Hkv, D, page, n, window, sinks = 2, 8, 2, 128, 32, 700, 150, 4
    q, k, v = _qkv(B, Hq, Hkv, n + 8, n + 8, D, BF, 5)
    table = A.rope_table(n + 8, D)
    kr = A.rope_apply(k, table)
    pages = -(-(n + 8) // page)
    kc, vc = (torch.zeros((B * pages, Hkv, page, D), dtype=BF, device="cuda") for _ in range(2))
    bt = torch.randperm(B * pages, device="cuda").int().reshape(B, pages)
    lens = lambda m: torch.full((B,), m, dtype=torch.int32, device="cuda")      # noqa: E731
    A.kv_append(k[:, :n].contiguous(), v[:, :n].contiguous(), kc, vc, bt, lens(n), table=table)
    for i in range(n, n + 8):
        A.kv_append(k[:, i:i + 1], v[:, i:i + 1], kc, vc, bt, lens(i + 1), table=table)
        o, lse = A.attention_paged(q[:, i:i + 1], kc, vc, bt, lens(i + 1), table=table, window=window, sinks=sinks)
        qr = A.rope_apply(q[:, :i + 1].contiguous(), table)
        w, wl = A.attention_window(qr, kr[:, :i + 1].contiguous(), v[:, :i + 1].contiguous(), window=window, sinks=sinks)
        # as above: the weights are rounded to bf16 on both sides, the outputs too
        bound = 2 * 2.0 ** -8 * (w[:, -1:].float().abs() + v.float().abs().max())
        assert bool(((o.float() - w[:, -1:].float()).abs() <= bound).all())
        assert float((lse[..., 0] - wl[..., -1]).abs().max()) <= 1e-4


def _call(fn=None, **kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, B=1, Hq=2, Hkv=2, Sq=300, Sk=300, D=64, scale=0.0, window=100, sinks=2,
             stream=None)
    a.update(kw)
    return (fn or A.attn_fwd_window)(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(window=0), A.ATTN_ERR_INVALID_ARG), (dict(window=-5), A.ATTN_ERR_INVALID_ARG),
    (dict(sinks=-1), A.ATTN_ERR_INVALID_ARG), (dict(q=None), A.ATTN_ERR_INVALID_ARG),
    (dict(v=P + 8), A.ATTN_ERR_INVALID_ARG), (dict(Hq=3), A.ATTN_ERR_INVALID_ARG),
    (dict(lse=P + 2), A.ATTN_ERR_INVALID_ARG), (dict(Sq=-1), A.ATTN_ERR_INVALID_ARG),
    (dict(D=96), A.ATTN_ERR_UNSUPPORTED), (dict(B=0), A.ATTN_OK), (dict(Sq=0), A.ATTN_OK),
])
def test_window_arguments(kw, code):
    A.lib()
    assert _call(**kw) == code and _call(A.attn_fwd_window_f16, **kw) == code


def test_window_python_refusals():
    q, k = torch.zeros(1, 8, 2, 64, dtype=BF), torch.zeros(1, 8, 2, 64, dtype=FP)
    for args in ((q, q, q), (q, k, q), (q.float(), q, q), (q[0], q, q)):
        with pytest.raises(ValueError):
            A.attention_window(*args, window=3)
