"""Pages out of range under long chunks of queries: hidden by the gathered pages as by the cache itself, so that the size
of the workspace, which picks the way, does not change the answer."""
import numpy as np
import pytest
import torch

import paged_ref as R
from test_paged import BF, DEV, FP, Cache, _i32, _rand, _status, _v_top
from transformer_attention_02_gb300 import attn as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(24, 2, 128, 16), (24, 2, 64, 128), (48, 4, 64, 32)])
def test_a_long_chunk_hides_pages_out_of_range(Hq, Hkv, D, page, e4m3):
    """The keys of a page out of range are hidden whichever way the call goes: rows that see no other get o = 0, lse =
    -inf. Both paths against the 64-bit form without those keys."""
    kv, ql, Sq, keys = [700, 130], [140, 130], 140, 8192
    c = Cache(2, Hkv, D, page, keys // page, BF, e4m3, seed=D + page)
    c.fill(0, kv[0], 0), c.fill(1, kv[1], 1)
    gone = [[1, 3, (kv[0] - 1) // page], [0]]               # the last page of one sequence, the first of the other
    table, n = c.table.clone(), 0
    for b in range(2):
        for j in gone[b]:
            table[b, j] = [-1, c.k.shape[0], -(1 << 31), 1 << 30][n]
            n += 1
    q = _rand((2, Sq, Hq, D), BF, 9)
    small = torch.empty(A.attn_paged_workspace_bytes(2, Hq, Hkv, Sq, D), dtype=torch.uint8, device=DEV)
    assert small.numel() < A.attn_paged_workspace_bytes(2, Hq, Hkv, Sq, D, keys)
    for ws in (None, small):
        o, lse = A.attention_paged(q, c.k, c.v, table, _i32(kv), q_lens=_i32(ql), workspace=ws, **c.scales)
        assert _status() == A.ATTN_ERR_BAD_INDEX
        for b in range(2):
            keep = np.array([t // page not in gone[b] for t in range(kv[b])])
            k, v = (R.tokens(x, s, c.table_np[b], kv[b], page)[keep] for x, s in ((c.k, c.ks), (c.v, c.vs)))
            pos = np.cumsum(keep)[kv[b] - ql[b]:] - 1       # of the last key left that a query sees (-1: none)
            assert b == 0 or pos[0] < 0
            want = R.attend(R.f64(q[b, :ql[b]]), k, v, pos, D ** -0.5, 0, 0)
            R.check_rows(R.f64(o[b, :ql[b]]), R.f64(lse[b, :, :ql[b]]), want, R.step(BF), R.step(BF), D, kv[b],
                         _v_top(c, c.table_np[b, :-(-kv[b] // page)]), f"{ws is None} b={b}")


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "f16"])
@pytest.mark.parametrize("D,page,window,sinks", [(128, 16, 200, 40), (64, 16, 33, 0), (64, 256, 600, 300)])
def test_the_paths_agree_on_bad_pages_in_a_window(D, page, window, sinks, dt):
    """Some pages out of range among the sinks, in the window and between them, ragged: by the gathered pages and by the
    cache itself, within the rounding of the weights."""
    kv, ql, Sq, Hq, Hkv, keys = [1500, 900, 0, 160], [160, 3, 0, 160], 160, 12, 4, 8192
    c = Cache(4, Hkv, D, page, keys // page, dt, False, seed=page)
    table = c.table.clone()
    for b in range(4):
        c.fill(b, kv[b], b)
        for j in range(0, -(-kv[b] // page), 3):
            table[b, j] = -1
    q = _rand((4, Sq, Hq, D), dt, 11)
    small = torch.empty(A.attn_paged_workspace_bytes(4, Hq, Hkv, Sq, D), dtype=torch.uint8, device=DEV)
    got = []
    for ws in (None, small):
        o, lse = torch.zeros_like(q), torch.zeros((4, Hq, Sq), device=DEV)
        A.attention_paged(q, c.k, c.v, table, _i32(kv), q_lens=_i32(ql), window=window, sinks=sinks, workspace=ws, out=o,
                          lse=lse, **c.scales)
        assert _status() == A.ATTN_ERR_BAD_INDEX
        got.append((o.double(), lse.double()))
    (o, lse), (o2, lse2) = got
    # the weights are rounded once on each side (half a step of sum p|v| <= max|v|), the outputs too
    top = float(torch.nan_to_num(c.v.double()).abs().max())
    assert float((o - o2).abs().max()) <= 2 * R.step(dt) * (top + float(o.abs().max())) + 1e-5
    none = lse == float("-inf")
    assert bool((none == (lse2 == float("-inf"))).all()) and bool(torch.isfinite(o).all())
    assert bool((o.permute(0, 2, 1, 3)[none] == 0).all())
    assert float((lse - lse2)[~none].abs().max()) <= 1e-4
