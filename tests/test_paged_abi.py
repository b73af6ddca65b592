"""Host-side checks of the paged cache's entry points (no GPU): every refusal happens before any device call, with
stand-in addresses that are never used."""
import pytest
import torch

from transformer_attention_02_gb300 import attn as A
from transformer_attention_02_gb300 import build as B

P = 0x10000


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return A.lib()


def _append(fn=None, **kw):
    a = dict(k=P, v=P, k_stride=128, v_stride=128, k_cache=P, v_cache=P, k_scale=P, v_scale=P, block_table=P, kv_lens=P,
             new_lens=None, B=2, S=3, Hkv=2, D=64, page=16, max_pages=4, n_pages=8, cache_kind=A.CACHE_E4M3,
             rope_table=None, max_pos=0, stream=None)
    a.update(kw)
    return (fn or A.attn_kv_append)(**a)


APPEND_BAD = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(k_scale=None), 1),
    (dict(v_scale=None), 1), (dict(block_table=None), 1), (dict(kv_lens=None), 1), (dict(k=P + 8), 1),
    (dict(v_cache=P + 4), 1), (dict(kv_lens=P + 2), 1), (dict(new_lens=P + 1), 1), (dict(k_stride=127), 1),
    (dict(k_stride=120), 1), (dict(v_stride=132), 1), (dict(B=-1), 1), (dict(S=-1), 1), (dict(Hkv=0), 1),
    (dict(page=8), 1), (dict(page=24), 1), (dict(page=512), 1), (dict(max_pages=0), 1), (dict(n_pages=0), 1),
    (dict(cache_kind=2), 1), (dict(D=96), 2), (dict(D=32), 2), (dict(rope_table=P + 4, max_pos=64), 1),
    (dict(rope_table=P, max_pos=0), 1), (dict(max_pages=1 << 27), 1), (dict(B=1 << 30, S=1 << 20), 1),
    (dict(B=0), 0), (dict(S=0), 0),
]


@pytest.mark.parametrize("kw,code", APPEND_BAD)
def test_append_arguments(kw, code):
    assert _append(**kw) == code and _append(A.attn_kv_append_f16, **kw) == code


def test_a_16_bit_cache_needs_no_scales():
    assert _append(k_scale=None, v_scale=None, cache_kind=A.CACHE_16BIT) not in (A.ATTN_OK, A.ATTN_ERR_INVALID_ARG)


def _attend(fn=None, **kw):
    a = dict(q=P, q_stride=256, k_cache=P, v_cache=P, k_scale=P, v_scale=P, block_table=P, kv_lens=P, q_lens=None, o=P,
             lse=P, B=2, Hq=4, Hkv=2, Sq=1, D=64, page=16, max_pages=4, n_pages=8, cache_kind=A.CACHE_E4M3, scale=0.0,
             window=0, sinks=0, rope_table=None, max_pos=0, workspace=P, workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    return (fn or A.attn_fwd_paged)(**a)


ATTEND_BAD = [
    (dict(q=None), 1), (dict(o=None), 1), (dict(lse=None), 1), (dict(k_cache=None), 1), (dict(k_scale=None), 1),
    (dict(block_table=None), 1), (dict(kv_lens=None), 1), (dict(q=P + 8), 1), (dict(o=P + 2), 1), (dict(lse=P + 2), 1),
    (dict(q_lens=P + 2), 1), (dict(q_stride=248), 1), (dict(q_stride=257), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1),
    (dict(Sq=-1), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(page=48), 1), (dict(cache_kind=-1), 1),
    (dict(D=80), 2), (dict(rope_table=P), 1), (dict(workspace=None), 1), (dict(workspace=P + 16), 1),
    (dict(workspace_bytes=1000), 1), (dict(B=1 << 24, max_pages=1 << 20), 1), (dict(Sq=1 << 30, Hq=4096), 1),
    (dict(B=0), 0), (dict(Sq=0), 0), (dict(Hq=0, q_stride=0), 0),
]


@pytest.mark.parametrize("kw,code", ATTEND_BAD)
def test_attention_arguments(kw, code):
    assert _attend(**kw) == code and _attend(A.attn_fwd_paged_f16, **kw) == code


def test_workspace_size():
    # 148 SMs assumed without a GPU: (B + 1) sequence offsets, then two parts of rows x (D + 2) FP32 per CTA; rows
    # come in blocks of 8, 16, 24 or 32, three CTAs an SM, two for blocks of 24 and 32 rows of 128
    assert A.attn_paged_workspace_bytes(16, 32, 8, 1, 128) == 256 + 148 * 3 * 2 * 8 * 130 * 4
    assert A.attn_paged_workspace_bytes(16, 32, 8, 4, 64) == 256 + 148 * 3 * 2 * 16 * 66 * 4
    assert A.attn_paged_workspace_bytes(1, 32, 1, 9, 64) == 256 + 148 * 3 * 2 * 32 * 66 * 4
    assert A.attn_paged_workspace_bytes(1, 32, 1, 9, 128) == 256 + 148 * 2 * 2 * 32 * 130 * 4
    # a short table bounds the CTAs: 8 segments of 5 units (577 keys), one more for sinks, and the schedule's lead
    assert A.attn_paged_workspace_bytes(1, 32, 8, 1, 128, 577) == 256 + 8 * (5 + 4) * 2 * 8 * 130 * 4
    assert A.attn_paged_workspace_bytes(16, 32, 8, 1, 128, 8192) == A.attn_paged_workspace_bytes(16, 32, 8, 1, 128)
    assert A.attn_paged_workspace_bytes(16, 32, 8, 1, 128, -1) == 0
    assert A.attn_paged_workspace_bytes(16, 32, 8, 128, 128, (1 << 30) + 1) == 0
    assert A.attn_paged_workspace_bytes(16, 32, 8, 128, 128, (1 << 32) + 16) == 0
    # long chunks (128 queries, 48 tiles): gathered keys and values, then the queries; else, or past 4 GiB, as above
    assert A.attn_paged_workspace_bytes(2, 32, 8, 128, 64, 1000 * 16) == 2 * (2 * 16000 * 8 * 64 * 2) + 2 * 128 * 32 * 64 * 2
    few = 256 + 148 * 3 * 2 * 32 * 66 * 4
    assert A.attn_paged_workspace_bytes(2, 32, 8, 128, 64) == few
    assert A.attn_paged_workspace_bytes(2, 32, 8, 127, 64, 1000 * 16) == few
    assert A.attn_paged_workspace_bytes(1, 32, 8, 256, 64, 1000 * 16) == few
    assert A.attn_paged_workspace_bytes(64, 32, 8, 128, 64, 1 << 20) == few + 256       # (66 offsets: 512 bytes)
    assert A.attn_paged_workspace_bytes(0, 32, 8, 1, 128) == 0
    assert A.attn_paged_workspace_bytes(1, 30, 8, 1, 128) == 0
    assert A.attn_paged_workspace_bytes(1, 32, 8, 1, 96) == 0


def test_status_string():
    assert A.attn_status_string(A.ATTN_ERR_BAD_INDEX) == "ATTN_ERR_BAD_INDEX"


def _t(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt)


def test_python_refusals():
    """Types, shapes and layouts the wrappers refuse before any call (host tensors reach no further than these checks)."""
    cache, f8 = _t(4, 2, 16, 64), torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s, table, lens = torch.ones(4, 2), torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q, k = _t(1, 1, 4, 64), _t(1, 1, 2, 64)

    def refused(match, f, *a, **kw):
        with pytest.raises(ValueError, match=match):
            f(*a, **kw)

    refused("needs its scales", A.attention_paged, q, f8, f8, table, lens)
    refused("has no scales", A.attention_paged, q, cache, cache, table, lens, k_scale=s, v_scale=s)
    refused("bf16 or fp16", A.attention_paged, q.float(), cache, cache, table, lens)
    refused("float8_e4m3fn or of", A.attention_paged, q.half(), cache, cache, table, lens)
    refused("contiguous", A.attention_paged, q, cache.transpose(2, 3), cache.transpose(2, 3), table, lens)
    refused("int32", A.attention_paged, q, cache, cache, table.long(), lens)
    refused("int32", A.attention_paged, q, cache, cache, table, lens.repeat(2))
    refused("table must be", A.attention_paged, q, cache, cache, table, lens, table=torch.zeros(8, 16, 2))
    refused("CUDA tensor", A.attention_paged, q, cache, cache, table, lens)
    refused("one type", A.kv_append, k, k.half(), cache, cache, table, lens)
    refused("Hkv and D", A.kv_append, _t(1, 1, 3, 64), _t(1, 1, 3, 64), cache, cache, table, lens)
    refused("CUDA tensor", A.kv_append, k, k, cache, cache, table, lens)
