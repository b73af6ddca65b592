"""Attention over a paged cache whose unseen keys are not there: pages between the sinks and the window that hold NaN,
have scales of NaN or infinity, or have left the table. Results and status are those of a cache where they are fine."""
import numpy as np
import pytest
import torch

from test_paged import BF, DEV, FP, Cache, _check_attention, _i32, _rand, _status
from transformer_attention_02_gb300 import attn as A

pytestmark = pytest.mark.gpu

GONE = [-1, 1 << 30, -(1 << 31)]


def _unseen(kv, ql, window, sinks):
    """True for the keys of a sequence that none of its ql queries sees."""
    j = np.arange(kv)
    return (j < kv - ql - window + 1) & (j >= sinks)


def _spoil(c, b, hidden):
    """NaN (16-bit values: infinity) into every unseen slot, NaN and infinity into the scales of pages without another;
    returns those pages' places in the table."""
    page, whole = c.page, []
    for j in range(-(-len(hidden) // page)):
        at, part = int(c.table_np[b, j]), hidden[j * page:(j + 1) * page]
        slots = torch.as_tensor(np.flatnonzero(part), device=DEV)
        if c.ks is None:
            c.k[at, :, slots] = float("nan")
            c.v[at, :, slots] = float("inf")
        else:
            c.k.view(torch.uint8)[at, :, slots] = 0x7F
            c.v.view(torch.uint8)[at, :, slots] = 0x7F
        if part.all() and len(part) == page:
            whole.append(j)
            if c.ks is not None:
                c.ks[at], c.vs[at] = (float("nan"), float("inf")) if j % 2 else (float("inf"), float("nan"))
    return whole


def _agree(case, dt, e4m3, workspaces, keys=0):
    """keys: width of the table, if wider than the longest sequence."""
    Hq, Hkv, D, page, kv, ql, Sq, window, sinks = case
    B = len(kv)
    c = Cache(B, Hkv, D, page, -(-max(*kv, keys) // page), dt, e4m3, seed=sum(kv))
    for b in range(B):
        c.fill(b, kv[b], b)
    q = _rand((B, Sq, Hq, D), dt, 7)
    kw = dict(q_lens=_i32(ql), window=window, sinks=sinks, **c.scales)

    def run(table, ws):
        o, lse = torch.zeros_like(q), torch.zeros((B, Hq, Sq), device=DEV)
        A.attention_paged(q, c.k, c.v, table, _i32(kv), out=o, lse=lse, workspace=ws, **kw)
        return o, lse, _status()

    clean = [run(c.table, ws) for ws in workspaces]
    for o, lse, status in clean:
        assert status == A.ATTN_OK
    if Sq < 128:                                                     # (the long chunks' own test checks those)
        _check_attention(c, q, q, *clean[0][:2], kv, ql, window, sinks, label=str(case))
    table, n = c.table.clone(), 0
    for b in range(B):
        for j in _spoil(c, b, _unseen(kv[b], ql[b], window, sinks)):
            table[b, j] = GONE[n % 3]
            n += 1
    assert n > 0
    for ws, want in zip(workspaces, clean):
        for t in (c.table, table):
            o, lse, status = run(t, ws)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
            assert status == A.ATTN_OK


CASES = [
    # Hq, Hkv, D, page, kv_lens, q_lens, Sq, window, sinks
    (8, 2, 128, 16, [700, 650], [1, 1], 1, 77, 4),           # one token; unseen pages beside the sinks' and the window's
    (8, 2, 128, 16, [370, 300], [1, 1], 1, 77, 4),           # the same over a short table
    (8, 2, 64, 32, [2000, 1333], [5, 2], 5, 300, 70),        # drafts: 20 rows
    (8, 1, 128, 64, [1500, 900], [3, 3], 3, 200, 0),         # 24 rows, no sinks
    (16, 2, 64, 16, [1001, 640], [2, 2], 2, 50, 17),         # 16 rows
    (4, 1, 64, 16, [1200, 400], [20, 20], 20, 130, 19),      # 80 rows: three row blocks
    (4, 4, 128, 128, [900, 515], [2, 1], 2, 140, 4),         # pages as long as a unit
]


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "f16"])
@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "H{}-{}_D{}_p{}_{}_{}_w{}s{}".format(*c[:6], *c[7:]))
def test_unseen_pages(case, e4m3, dt):
    _agree(case, dt, e4m3, [None])


CHUNKS = [
    (24, 2, 128, 16, [700, 650], [130, 130], 130, 200, 4),
    (24, 2, 128, 64, [1100, 333], [200, 7], 200, 300, 0),     # a chunk beside a few tokens
    (12, 4, 64, 16, [1000, 900, 0, 777], [128, 140, 0, 1], 140, 129, 140),
    (24, 8, 64, 256, [1500, 1027], [128, 130], 130, 290, 19),
]


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "f16"])
@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "H{}-{}_D{}_p{}_{}_{}_w{}s{}".format(*c[:6], *c[7:]))
def test_unseen_pages_of_a_long_chunk(case, e4m3, dt):
    """By the gathered pages (the default workspace) and, with the small workspace, by the cache itself."""
    Hq, Hkv, D, page, kv, _, Sq = case[:7]
    keys = 8192                                             # (a table for which the gathered tensors are the larger scratch)
    small = A.attn_paged_workspace_bytes(len(kv), Hq, Hkv, Sq, D)
    assert small < A.attn_paged_workspace_bytes(len(kv), Hq, Hkv, Sq, D, keys)
    _agree(case, dt, e4m3, [None, torch.empty(small, dtype=torch.uint8, device=DEV)], keys)
