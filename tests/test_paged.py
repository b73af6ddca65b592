"""The paged key/value cache on the GPU: appending (rotation, 8-bit blocks, what stays untouched) and attention over
the cache, against the plain 64-bit forms of paged_ref; bounds are derived there and beside each test."""
import numpy as np
import pytest
import torch

import paged_ref as R
from transformer_attention_02_gb300 import attn as A

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")
BF, FP = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _status():
    return A.attn_last_status(torch.cuda.current_stream().cuda_stream)


def _rand(shape, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dt).to(DEV)


class Cache:
    """A cache with pages in shuffled order; 16-bit slots start as NaN, 8-bit ones as NaN codes."""

    def __init__(self, B, Hkv, D, page, max_pages, dt, e4m3, seed=0, spare=2):
        n = B * max_pages + spare
        shape = (n, Hkv, page, D)
        if e4m3:
            self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
                              for _ in range(2))
            self.ks, self.vs = (torch.full((n, Hkv), float("nan"), device=DEV) for _ in range(2))
        else:
            self.k, self.v = (torch.full(shape, float("nan"), dtype=dt, device=DEV) for _ in range(2))
            self.ks = self.vs = None
        perm = np.random.RandomState(seed).permutation(n)[:B * max_pages].reshape(B, max_pages)
        self.table_np = perm.astype(np.int32)
        self.table = _i32(self.table_np.tolist())
        self.page = page

    @property
    def scales(self):
        return dict(k_scale=self.ks, v_scale=self.vs)

    def fill(self, b, n, seed):
        """Random content for the first n tokens of sequence b; the rest stays NaN."""
        page, (_, Hkv, _, D) = self.page, self.k.shape
        g = np.random.RandomState(seed)
        for t, s in ((self.k, self.ks), (self.v, self.vs)):
            for j in range(-(-n // page)):
                m = min(page, n - j * page)
                x = torch.tensor(g.randn(Hkv, m, D) * 2.0 ** g.randint(-2, 3), dtype=torch.float32, device=DEV)
                at = int(self.table_np[b, j])
                if s is None:
                    t[at, :, :m] = x.to(t.dtype)
                else:
                    sc = torch.tensor([R.block_scale(float(x[h].abs().max())) for h in range(Hkv)], device=DEV)
                    s[at] = sc
                    t.view(torch.uint8)[at, :, :m] = (x / sc[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _v_top(c, ids):
    ids = torch.as_tensor(ids.astype(np.int64), device=DEV)
    if c.vs is not None:
        return float(torch.nan_to_num(c.vs[ids]).max()) * 448.0
    return float(torch.nan_to_num(c.v[ids].float()).abs().max())


def _check_attention(c, q, q_rot, o, lse, kv, ql, window=0, sinks=0, scale=None, label=""):
    B, Sq, Hq, D = q.shape
    p_step = R.step(q.dtype) if c.ks is None else R.step(FP)
    sc = D ** -0.5 if scale is None else scale
    for b in range(B):
        n, L = ql[b], kv[b]
        if n == 0:
            continue
        pos = np.arange(L - n, L)
        k, v = (R.tokens(x, s, c.table_np[b], L, c.page) for x, s in ((c.k, c.ks), (c.v, c.vs)))
        want = R.attend(R.f64(q_rot[b, :n]), k, v, pos, sc, window, sinks)
        R.check_rows(R.f64(o[b, :n]), R.f64(lse[b, :, :n]), want, R.step(q.dtype), p_step, D, L,
                     _v_top(c, c.table_np[b, :max(1, -(-L // c.page))]), f"{label} b={b}")


# ------------------------------------------------------------------ append

APPEND = [
    # Hkv, D, page, tokens before per sequence, new per sequence, S, rope
    (8, 128, 64, [0], [1], 1, True),                       # the very first token
    (2, 64, 16, [15, 16, 17, 0], [1, 1, 1, 0], 1, True),   # last slot, fresh page, second slot, idle sequence
    (3, 128, 32, [5, 0, 31], [70, 33, 1], 70, True),       # over several pages, ragged
    (1, 64, 256, [100], [200], 200, False),                # not rotated
    (4, 128, 16, [0, 7], [16, 9], 16, True),               # pages that end exactly full
]


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "f16"])
@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"H{c[0]}_D{c[1]}_p{c[2]}_{c[3]}+{c[4]}")
def test_append(case, dt, e4m3):
    Hkv, D, page, before, new, S, rope = case
    B = len(before)
    kv = [p + n for p, n in zip(before, new)]
    max_pages = -(-max(kv) // page) + 1
    c = Cache(B, Hkv, D, page, max_pages, dt, e4m3, seed=sum(kv))
    for b in range(B):
        c.fill(b, before[b], 100 + b)
    was = {n: getattr(c, n).clone() for n in ("k", "v")}
    was_s = None if not e4m3 else {"k": c.ks.clone(), "v": c.vs.clone()}
    k, v = _rand((B, S, Hkv, D), dt, 1, 3.0), _rand((B, S, Hkv, D), dt, 2, 0.7)
    table = A.rope_table(max_pages * page, D) if rope else None
    A.kv_append(k, v, c.k, c.v, c.table, _i32(kv), new_lens=_i32(new), table=table, **c.scales)
    assert _status() == A.ATTN_OK
    touched = {"k": torch.zeros(c.k.shape[:3], dtype=torch.bool, device=DEV)}
    for name, x, cache, scale in (("k", k, c.k, c.ks), ("v", v, c.v, c.vs)):
        changed = torch.zeros(cache.shape[:3], dtype=torch.bool, device=DEV)
        own_block = torch.zeros(cache.shape[:2], dtype=torch.bool, device=DEV)
        for b in range(B):
            pos = np.arange(before[b], kv[b])
            x64 = R.f64(x[b, :new[b]])
            want = R.rotate(x64, pos) if (rope and name == "k") else x64
            # FP32 rotation: two products and a sum, each off by 2^-24 of the pair, and a table entry off by 2^-25
            pair = np.repeat(np.abs(x64[..., 0::2]) + np.abs(x64[..., 1::2]), 2, axis=-1) * 2.0 ** -22
            for j in sorted(set((pos // page).tolist())):
                at, sel = int(c.table_np[b, j]), pos // page == j
                slots = torch.as_tensor(pos[sel] % page, device=DEV)
                for h in range(Hkv):
                    got = R.f64(cache.float()[at, h][slots])
                    w, e = want[sel][:, h], pair[sel][:, h]
                    if e4m3:
                        own_block[at, h] = True
                        s = float(scale[at, h])
                        need = R.block_scale(np.abs(w).max())
                        old = int(pos[sel][0]) % page
                        if old:
                            s0 = float(was_s[name][at, h])
                            need = max(need, s0)
                            # earlier codes: moved by a power of two, exact but for half a subnormal step
                            o0 = R.f64(was[name].float()[at, h, :old]) * s0
                            o1 = R.f64(cache.float()[at, h, :old]) * s
                            assert np.all(np.abs(o1 - o0) <= (0 if s == s0 else 2.0 ** -10 * s))
                            changed[at, h, :old] = s != s0
                        assert s == need, (name, b, j, h, s, need)
                        tol = R.step(torch.float8_e4m3fn) * np.abs(w) + 2.0 ** -10 * s + e
                        got = got * s
                    else:
                        tol = R.step(dt) * np.abs(w) + (e if name == "k" and rope else 0) + 2.0 ** -25
                    assert np.all(np.abs(got - w) <= tol), (name, b, j, h)
                changed[at, :, slots] = True
        # everything else is as it was, byte for byte
        same = cache.view(torch.uint8 if e4m3 else torch.int16) == was[name].view(torch.uint8 if e4m3 else torch.int16)
        assert bool(same[~changed].all())
        if e4m3:
            assert bool((scale.view(torch.int32) == was_s[name].view(torch.int32))[~own_block].all())


def test_append_grows_a_block_scale_and_keeps_earlier_values():
    """Token magnitudes that double sixteen times within one page: every earlier code survives each growth until it
    enters the subnormal range, where it loses at most half a subnormal step a growth."""
    c = Cache(1, 1, 64, 32, 1, BF, True)
    x = torch.stack([_rand((1, 64), BF, i) * 2.0 ** i for i in range(16)])[None]       # (1, 16, 1, 64)
    for i in range(16):
        A.kv_append(x[:, i:i + 1], x[:, i:i + 1], c.k, c.v, c.table, _i32([i + 1]), **c.scales)
    s = float(c.vs[c.table_np[0, 0], 0])
    got = R.f64(c.v.float()[c.table_np[0, 0], 0, :16]) * s
    want = R.f64(x[0, :, 0])
    # first quantisation, then half a subnormal step of each scale up to the last (their sum is below the last's step)
    assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * s)
    assert s == R.block_scale(np.abs(want).max())


def test_append_of_zeros_infinities_and_nan():
    c = Cache(1, 1, 64, 16, 1, BF, True)
    x = torch.zeros((1, 3, 1, 64), dtype=BF, device=DEV)
    x[0, 1, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1.0])
    A.kv_append(x[:, :1], x[:, :1], c.k, c.v, c.table, _i32([1]), **c.scales)
    at = int(c.table_np[0, 0])
    assert float(c.ks[at, 0]) == 2.0 ** -100 and bool((c.k.float()[at, 0, 0] == 0).all())
    A.kv_append(x, x, c.k, c.v, c.table, _i32([3]), **c.scales)
    assert float(c.ks[at, 0]) == R.block_scale(1.0) == float(c.vs[at, 0])
    got = (c.k.float() * c.ks[:, :, None, None])[at, 0, 1, :4].cpu()
    top = 448.0 * R.block_scale(1.0)
    assert got[0] == top and got[1] == -top and torch.isnan(got[2]) and got[3] == 1.0


def test_append_reads_slices_of_a_packed_projection():
    B, S, Hq, Hkv, D = 3, 5, 4, 2, 64
    qkv = _rand((B, S, (Hq + 2 * Hkv) * D), BF, 3)
    k = qkv[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    v = qkv[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D))
    one, two = (Cache(B, Hkv, D, 16, 2, BF, True) for _ in range(2))
    table, kv = A.rope_table(32, D), _i32([9, 20, 5])
    A.kv_append(k, v, one.k, one.v, one.table, kv, table=table, **one.scales)
    A.kv_append(k.contiguous(), v.contiguous(), two.k, two.v, two.table, kv, table=table, **two.scales)
    assert torch.equal(one.k.view(torch.uint8), two.k.view(torch.uint8))
    assert torch.equal(one.v.view(torch.uint8), two.v.view(torch.uint8))
    last = k[:, 2:3], v[:, 2:3]                                            # one token each: the batch stride leads
    A.kv_append(*last, one.k, one.v, one.table, kv, table=table, **one.scales)
    A.kv_append(*(t.contiguous() for t in last), two.k, two.v, two.table, kv, table=table, **two.scales)
    assert torch.equal(one.k.view(torch.uint8), two.k.view(torch.uint8))


def test_append_leaves_out_what_is_out_of_range():
    B, Hkv, D, page = 4, 2, 64, 16
    c = Cache(B, Hkv, D, page, 2, FP, False)
    c.table[1, 0] = c.k.shape[0]                                           # a page past the cache
    c.table[2, 0] = -1
    k = _rand((B, 3, Hkv, D), FP, 5)
    was = c.k.clone()
    A.kv_append(k, k, c.k, c.v, c.table, _i32([3, 3, 3, 33]))                # the last: longer than its table
    assert _status() == A.ATTN_ERR_BAD_INDEX and _status() == A.ATTN_OK
    at = int(c.table_np[0, 0])
    assert torch.equal(c.k[at, :, :3], k[0].transpose(0, 1))
    was[at] = c.k[at]
    assert torch.equal(c.k.view(torch.int16), was.view(torch.int16))
    A.kv_append(k, k, c.k, c.v, c.table, _i32([3, 0, 0, 2]), new_lens=_i32([0, 0, 0, 3]))   # more new than there are
    assert _status() == A.ATTN_ERR_BAD_INDEX
    assert torch.equal(c.k.view(torch.int16), was.view(torch.int16))


# --------------------------------------------------------------- attention

ATTEND = [
    # Hq, Hkv, D, page, kv_lens, q_lens, Sq, window, sinks
    (8, 2, 128, 64, [1], [1], 1, 0, 0),                            # one key
    (32, 8, 128, 64, [500, 0, 129], [1, 1, 1], 1, 0, 0),           # an empty sequence among others
    (4, 4, 64, 16, [77, 16, 17], [1, 1, 1], 1, 0, 0),              # MHA: one row a head
    (7, 1, 128, 32, [1000, 31], [1, 1], 1, 0, 0),                  # a group of seven, MQA
    (16, 1, 64, 128, [700], [1], 1, 0, 0),                         # sixteen rows
    (64, 2, 128, 16, [300, 45], [1, 1], 1, 0, 0),                  # 32 rows
    (6, 2, 128, 64, [900, 40, 5], [5, 3, 5], 5, 0, 0),             # several queries a sequence, ragged, 15 rows
    (8, 2, 64, 32, [333, 20], [20, 20], 20, 0, 0),                 # 80 rows: three row blocks
    (4, 1, 128, 16, [3, 9], [5, 9], 5 + 4, 0, 0),                  # more queries than keys: rows without a key
    (8, 2, 128, 64, [2000, 1, 130], [1, 1, 1], 1, 100, 4),         # window and sinks, a gap between them
    (8, 2, 128, 64, [2000, 600], [6, 2], 6, 300, 150),             # sinks past a unit
    (4, 2, 64, 16, [513, 40], [3, 3], 3, 1, 0),                    # each query sees itself alone
    (4, 2, 64, 256, [513, 40], [3, 0], 3, 1000000, 2),             # a window longer than the cache; an idle sequence
]


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "f16"])
@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "H{}-{}_D{}_p{}_{}_{}_w{}s{}".format(*c[:6], *c[7:]))
def test_attention(case, dt, e4m3):
    """Every slot no key occupies holds NaN, so a read of one shows."""
    Hq, Hkv, D, page, kv, ql, Sq, window, sinks = case
    B = len(kv)
    c = Cache(B, Hkv, D, page, -(-max(kv) // page) + 1, dt, e4m3, seed=sum(kv))
    for b in range(B):
        c.fill(b, kv[b], b)
    q = _rand((B, Sq, Hq, D), dt, 7)
    o = torch.full_like(q, 5.0)
    lse = torch.full((B, Hq, Sq), 5.0, device=DEV)
    kw = dict(q_lens=_i32(ql), window=window, sinks=sinks, **c.scales)
    A.attention_paged(q, c.k, c.v, c.table, _i32(kv), out=o, lse=lse, **kw)
    assert _status() == A.ATTN_OK
    for b in range(B):                                              # rows behind the last query are left alone
        assert bool((o[b, ql[b]:] == 5.0).all()) and bool((lse[b, :, ql[b]:] == 5.0).all())
    _check_attention(c, q, q, o, lse, kv, ql, window, sinks, label=str(case))
    o2, lse2 = A.attention_paged(q, c.k, c.v, c.table, _i32(kv), out=o.clone(), lse=lse.clone(), **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)            # and the same bits every time


@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
def test_attention_rotates_the_queries(e4m3):
    kv, ql, Hq, Hkv, D = [300, 41, 3], [4, 4, 2], 8, 2, 128
    c = Cache(3, Hkv, D, 32, 11, BF, e4m3)
    for b in range(3):
        c.fill(b, kv[b], b)
    q, table = _rand((3, 4, Hq, D), BF, 8), A.rope_table(352, D)
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32(kv), q_lens=_i32(ql), table=table, **c.scales)
    rot = q.clone()
    for b in range(3):
        rot[b, :ql[b]] = A.rope_apply(q[b:b + 1, :ql[b]].contiguous(), table, pos0=kv[b] - ql[b])[0]
    _check_attention(c, q, rot, o, lse, kv, ql, label="rotated")


@pytest.mark.parametrize("mag", [1e-20, 1e-5, 3e4])
def test_attention_with_queries_of_any_magnitude(mag):
    """bf16 queries far outside fp16's range over an 8-bit cache; the scale brings the logits back to order one."""
    c = Cache(1, 2, 64, 16, 20, BF, True)
    c.fill(0, 300, 3)
    q = _rand((1, 1, 4, 64), BF, 9, mag)
    q[0, 0, 3] = 0
    sc = 0.1 / mag
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([300]), scale=sc, **c.scales)
    _check_attention(c, q, q, o, lse, [300], [1], scale=float(np.float32(sc)), label=str(mag))


def test_attention_with_one_dominant_key_late_in_a_long_cache():
    """The running maximum jumps by far more than the lazy threshold on the last page, and value scales differ by 2^40
    between pages."""
    c = Cache(1, 1, 128, 64, 64, BF, True)
    c.fill(0, 4000, 4)
    for j in range(63):
        at = int(c.table_np[0, j])
        c.vs[at] *= 2.0 ** ((j * 7) % 41 - 20)
    q = _rand((1, 1, 8, 128), BF, 10, 6.0)
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([4000]), **c.scales)
    _check_attention(c, q, q, o, lse, [4000], [1], label="dominant")


def test_attention_never_reads_hidden_values():
    """Keys and values before the window hold NaN: one query a sequence, so no query sees them."""
    c = Cache(2, 2, 128, 64, 12, FP, False)
    for b, n in enumerate((700, 650)):
        c.fill(b, n, b)
    q = _rand((2, 1, 4, 128), FP, 11)
    clean = A.attention_paged(q, c.k, c.v, c.table, _i32([700, 650]), window=77, sinks=3)
    for b, n in enumerate((700, 650)):
        for j in range(3, n - 77):
            c.k[int(c.table_np[b, j // 64]), :, j % 64] = float("nan")
            c.v[int(c.table_np[b, j // 64]), :, j % 64] = float("inf")
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([700, 650]), window=77, sinks=3)
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


def test_attention_hides_pages_out_of_range():
    c = Cache(2, 2, 64, 16, 4, FP, False)
    c.fill(0, 64, 0), c.fill(1, 64, 1)
    q = _rand((2, 1, 4, 64), FP, 12)
    kv = _i32([64, 64])
    c.table[0, 1] = c.k.shape[0] + 5
    o, lse = A.attention_paged(q, c.k, c.v, c.table, kv)
    assert _status() == A.ATTN_ERR_BAD_INDEX and _status() == A.ATTN_OK
    k, v = (R.tokens(x, None, c.table_np[0], 64, 16)[np.r_[0:16, 32:64]] for x in (c.k, c.v))
    want = R.attend(R.f64(q[0]), k, v, np.array([47]), 64 ** -0.5, 0, 0)
    R.check_rows(R.f64(o[0]), R.f64(lse[0]), want, R.step(FP), R.step(FP), 64, 64, _v_top(c, c.table_np[0]), "hidden page")
    # a length past the table is cut to it, a negative one to nothing
    c.table[0, 1] = int(c.table_np[0, 1])
    full = A.attention_paged(q, c.k, c.v, c.table, kv)
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([1 << 30, -4]))
    assert _status() == A.ATTN_ERR_BAD_INDEX
    assert torch.equal(o[0], full[0][0]) and bool((o[1] == 0).all()) and bool((lse[1] == float("-inf")).all())


def test_sequences_may_share_read_pages():
    c = Cache(2, 2, 64, 16, 4, BF, True)
    c.fill(0, 60, 0)
    c.table[1] = c.table[0]
    q = _rand((1, 1, 4, 64), BF, 13).expand(2, -1, -1, -1).contiguous()
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([60, 60]), **c.scales)
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes a tensor; the sequence's pages are its last ones."""
    Hkv, page, D = 8, 256, 128
    n = (1 << 32) // (Hkv * page * D) + 40
    k = torch.empty((n, Hkv, page, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    v = torch.empty_like(k.view(torch.uint8)).view(torch.float8_e4m3fn)
    ks, vs = torch.zeros((n, Hkv), device=DEV), torch.zeros((n, Hkv), device=DEV)
    table, kv = _i32([[n - 1, n - 3]]), _i32([400])
    x = _rand((1, 400, Hkv, D), BF, 14)
    A.kv_append(x, x, k, v, table, kv, k_scale=ks, v_scale=vs)
    q = _rand((1, 1, Hkv, D), BF, 15)
    o, lse = A.attention_paged(q, k, v, table, kv, k_scale=ks, v_scale=vs)
    small = [torch.stack([t[n - 1], t[n - 3]]).contiguous() for t in (k.view(torch.uint8), v.view(torch.uint8), ks, vs)]
    o2, lse2 = A.attention_paged(q, small[0].view(torch.float8_e4m3fn), small[1].view(torch.float8_e4m3fn),
                                 _i32([[0, 1]]), kv, k_scale=small[2], v_scale=small[3])
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and bool(torch.isfinite(lse).all())


def test_large_ragged_batch_over_many_ctas():
    """More segments than CTAs, lengths from 0 to several units, against a per-sequence call of its own."""
    B, Hkv, Hq, D, page = 300, 2, 8, 64, 16
    kv = [(37 * b) % 400 for b in range(B)]
    c = Cache(B, Hkv, D, page, 26, BF, True)
    c.k.view(torch.uint8).random_(0, 0x7E), c.v.view(torch.uint8).random_(0, 0x7E)
    c.ks.uniform_(0.001, 0.01), c.vs.uniform_(0.001, 0.01)
    q = _rand((B, 1, Hq, D), BF, 16)
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32(kv), **c.scales)
    for b in range(0, B, 23):
        _check_attention(_Row(c, b), q[b:b + 1], q[b:b + 1], o[b:b + 1], lse[b:b + 1], [kv[b]], [1], label=f"row {b}")


class _Row:
    def __init__(self, c, b):
        self.k, self.v, self.ks, self.vs, self.page, self.table_np = c.k, c.v, c.ks, c.vs, c.page, c.table_np[b:b + 1]


# ------------------------------------------------------------ used together

def test_graph_of_a_decode_step_replays_as_lengths_and_pages_change():
    B, Hq, Hkv, D, page, P = 3, 8, 2, 128, 16, 6
    c = Cache(B, Hkv, D, page, P, BF, True)
    table, kv = A.rope_table(P * page, D), _i32([0] * B)
    x = [_rand((B, 40, H, D), BF, 20 + i) for i, H in enumerate((Hq, Hkv, Hkv))]
    q, k, v = (torch.empty((B, 1, t.shape[2], D), dtype=BF, device=DEV) for t in x)
    out, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device=DEV)
    ws = torch.empty(A.attn_paged_workspace_bytes(B, Hq, Hkv, 1, D), dtype=torch.uint8, device=DEV)

    def step():
        A.kv_append(k, v, c.k, c.v, c.table, kv, table=table, **c.scales)
        A.attention_paged(q, c.k, c.v, c.table, kv, table=table, out=out, lse=lse, workspace=ws, **c.scales)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):                                        # first use: module loading, outside the capture
        kv.fill_(1), q.zero_(), k.zero_(), v.zero_()
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(40):
        for a, b in zip((q, k, v), x):
            a.copy_(b[:, i:i + 1])
        kv.fill_(i + 1)
        g.replay()
    torch.cuda.synchronize()
    assert _status() == A.ATTN_OK
    rot = torch.stack([A.rope_apply(q[b:b + 1], table, pos0=39)[0] for b in range(B)])
    _check_attention(c, q, rot, out, lse, [40] * B, [1] * B, label="graph")
    eager = Cache(B, Hkv, D, page, P, BF, True)
    for i in range(40):
        A.kv_append(x[1][:, i:i + 1], x[2][:, i:i + 1], eager.k, eager.v, eager.table, _i32([i + 1] * B), table=table,
                    **eager.scales)
    o2, l2 = A.attention_paged(q, eager.k, eager.v, eager.table, _i32([40] * B), table=table, **eager.scales)
    assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_side_stream():
    c = Cache(1, 2, 64, 16, 8, BF, True)
    c.fill(0, 100, 0)
    q = _rand((1, 1, 4, 64), BF, 30)
    want = A.attention_paged(q, c.k, c.v, c.table, _i32([100]), **c.scales)
    s, kv = torch.cuda.Stream(), _i32([100])
    torch.cuda.synchronize()
    o, lse = A.attention_paged(q, c.k, c.v, c.table, kv, stream=s, **c.scales)
    assert A.attn_last_status(s.cuda_stream) == A.ATTN_OK
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
def test_prompt_then_decode_steps(e4m3):
    """A prompt enters the cache in two chunks, then tokens one at a time; each step's attention is checked over what the
    cache holds, and with a 16-bit cache the prompt's against attention() on the contiguous rotated tensors."""
    B, Hq, Hkv, D, page, n = 2, 8, 2, 128, 32, 150
    c = Cache(B, Hkv, D, page, 6, BF, e4m3)
    table = A.rope_table(6 * page, D)
    q, k, v = (_rand((B, n, H, D), BF, 40 + i) for i, H in enumerate((Hq, Hkv, Hkv)))
    at, outs = 0, []
    for m in (70, 50) + (1,) * 30:
        kv = _i32([at + m] * B)
        A.kv_append(k[:, at:at + m].contiguous(), v[:, at:at + m].contiguous(), c.k, c.v, c.table, kv, table=table,
                    **c.scales)
        qs = q[:, at:at + m].contiguous()
        o, lse = A.attention_paged(qs, c.k, c.v, c.table, kv, table=table, **c.scales)
        if m > 1 or at == n - 1:
            _check_attention(c, qs, A.rope_apply(qs, table, pos0=at), o, lse, [at + m] * B, [m] * B, label=f"at {at}")
        outs.append(o)
        at += m
    if not e4m3:
        dense, _ = A.attention(A.rope_apply(q, table), A.rope_apply(k, table), v, causal=True)
        # the two paths round the same weights to bf16 separately: 2^-8 of sum p|v| each, and the outputs once each
        d = (torch.cat(outs, 1).float() - dense.float()).abs()
        bound = 2 * 2.0 ** -8 * dense.float().abs() + 2 * (2.0 ** -8 + 2.0 ** -14) * v.float().abs().amax()
        assert bool((d <= bound).all())


def test_calls_that_may_overlap_do_not_share_a_workspace():
    """Without a workspace argument: captured calls, side streams and threads use scratch of their own, so results are
    those of calls made one after the other."""
    import threading

    c = Cache(4, 2, 128, 64, 40, BF, True)
    for b in range(4):
        c.fill(b, 2500 - 100 * b, b)
    kv = [_i32([2500, 2400, 2300, 2200]), _i32([2000, 1, 1999, 64])]
    q = [_rand((4, 1, 8, 128), BF, 60 + i) for i in range(2)]
    want = [A.attention_paged(q[i], c.k, c.v, c.table, kv[i], **c.scales) for i in range(2)]
    # two graphs captured alike, replayed side by side
    outs, graphs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(A.attention_paged(q[i], c.k, c.v, c.table, kv[i], **c.scales))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    # two threads on the default stream, and a side stream beside them
    bad = []

    def loop(i, stream):
        for _ in range(50):
            o, l = A.attention_paged(q[i], c.k, c.v, c.table, kv[i], stream=stream, **c.scales)
            (stream or torch.cuda.current_stream()).synchronize()
            if not (torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])):
                bad.append(i)

    threads = [threading.Thread(target=loop, args=a) for a in ((0, None), (1, None), (1, streams[0]))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
@pytest.mark.parametrize("Hq,Hkv,D,Sq", [(8, 2, 64, 5), (8, 2, 128, 5), (3, 1, 64, 7), (4, 2, 128, 16), (8, 1, 64, 9)])
def test_row_blocks_of_24_and_32(Hq, Hkv, D, Sq, e4m3):
    """20, 21, 32 and 72 query rows a K/V head, over more keys than one CTA takes."""
    kv = [3000, Sq]
    c = Cache(2, Hkv, D, 64, 48, BF, e4m3)
    for b in range(2):
        c.fill(b, kv[b], b)
    q = _rand((2, Sq, Hq, D), BF, 70)
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32(kv), **c.scales)
    _check_attention(c, q, q, o, lse, kv, [Sq, Sq], label="row blocks")


def test_batches_past_256_sequences_and_many_segments_a_cta():
    """The merge reads the schedule from the workspace past 256 sequences; segments shorter and longer than a CTA's
    range, with the lead that the schedule gives each when there are many."""
    B, Hkv, Hq, D, page = 700, 4, 4, 64, 16
    kv = [(977 * b) % 1500 for b in range(B)]
    pages = 100
    n = 5000
    k, v = (torch.randint(0, 0x7E, (n, Hkv, page, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
            for _ in range(2))
    ks, vs = (torch.rand((n, Hkv), device=DEV) * 0.01 for _ in range(2))
    table = torch.randint(0, n, (B, pages), dtype=torch.int32, device=DEV)
    q = _rand((B, 1, Hq, D), BF, 80)
    o, lse = A.attention_paged(q, k, v, table, _i32(kv), k_scale=ks, v_scale=vs)
    row = object.__new__(_Row)
    row.k, row.v, row.ks, row.vs, row.page = k, v, ks, vs, page
    for b in range(0, B, 41):
        row.table_np = table[b:b + 1].cpu().numpy()
        _check_attention(row, q[b:b + 1], q[b:b + 1], o[b:b + 1], lse[b:b + 1], [kv[b]], [1], label=f"row {b}")


# ------------------------------------------------------- long chunks of queries

CHUNKS = [
    # Hq, Hkv, D, page, kv_lens, q_lens, Sq, window, sinks, rope
    (48, 8, 128, 64, [128], [128], 128, 0, 0, False),               # a prompt of its own
    (8, 2, 64, 16, [700, 130, 0, 40], [300, 130, 0, 7], 300, 0, 0, True),    # ragged; tiles without a query
    (12, 4, 128, 32, [1000, 333], [200, 333], 333, 150, 5, True),   # window and sinks
    (8, 1, 64, 256, [100, 600], [140, 600], 600, 0, 0, False),      # more queries than keys: rows without one
    (24, 8, 128, 16, [401, 500], [128, 200], 200, 129, 140, True),  # sinks over two blocks
]


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "f16"])
@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: "H{}-{}_D{}_p{}_{}_{}_w{}s{}".format(*c[:6], *c[7:9]))
def test_long_chunks(case, dt, e4m3):
    """By the gathered pages (the default workspace) and, with the small workspace, by the cache itself."""
    Hq, Hkv, D, page, kv, ql, Sq, window, sinks, rope = case
    B, pages = len(kv), -(-max(max(kv), Sq) // page) + 1
    c = Cache(B, Hkv, D, page, pages, dt, e4m3, seed=sum(kv))
    for b in range(B):
        c.fill(b, kv[b], b)
    q = _rand((B, Sq, Hq, D), dt, 90)
    table = A.rope_table(pages * page, D) if rope else None
    rot = q.clone()
    for b in range(B):
        if rope and ql[b]:
            rot[b, :ql[b]] = A.rope_apply(q[b:b + 1, :ql[b]].contiguous(), table, pos0=kv[b] - ql[b])[0]
    small = torch.empty(A.attn_paged_workspace_bytes(B, Hq, Hkv, Sq, D), dtype=torch.uint8, device=DEV)
    full = A.attn_paged_workspace_bytes(B, Hq, Hkv, Sq, D, pages * page)
    assert full >= 2 * B * pages * page * Hkv * D * 2
    # the gathered path rounds the weights to the queries' type, the other one to fp16 over an 8-bit cache; a workspace
    # that holds the gathered tensors takes the first
    by_cache = R.step(dt) if c.ks is None or small.numel() >= full else R.step(FP)
    for ws, p_step in ((None, R.step(dt)), (small, by_cache)):
        o, lse = torch.full_like(q, 5.0), torch.full((B, Hq, Sq), 5.0, device=DEV)
        A.attention_paged(q, c.k, c.v, c.table, _i32(kv), q_lens=_i32(ql), table=table, window=window, sinks=sinks, out=o,
                          lse=lse, workspace=ws, **c.scales)
        assert _status() == A.ATTN_OK
        for b in range(B):
            assert bool((o[b, ql[b]:] == 5.0).all()) and bool((lse[b, :, ql[b]:] == 5.0).all())
            if ql[b]:
                pos = np.arange(kv[b] - ql[b], kv[b])
                k, v = (R.tokens(x, s, c.table_np[b], kv[b], page) for x, s in ((c.k, c.ks), (c.v, c.vs)))
                want = R.attend(R.f64(rot[b, :ql[b]]), k, v, pos, D ** -0.5, window, sinks)
                R.check_rows(R.f64(o[b, :ql[b]]), R.f64(lse[b, :, :ql[b]]), want, R.step(dt), p_step, D, kv[b],
                             _v_top(c, c.table_np[b, :max(1, -(-kv[b] // page))]), f"{case} {ws is None} b={b}")


def test_long_chunk_leaves_out_what_is_out_of_range():
    c = Cache(2, 2, 64, 16, 20, FP, False)
    c.fill(0, 300, 0), c.fill(1, 300, 1)
    q = _rand((2, 128, 24, 64), FP, 91)
    want = A.attention_paged(q, c.k, c.v, c.table, _i32([300, 300]))
    c.table[1, 3] = -7
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([300, 300]))
    assert _status() == A.ATTN_ERR_BAD_INDEX and bool(torch.isfinite(o).all())
    assert torch.equal(o[0], want[0][0]) and torch.equal(lse[0], want[1][0])
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([-1, 1 << 29]), q_lens=_i32([128, 500]))
    assert _status() == A.ATTN_ERR_BAD_INDEX
    assert bool((o[0] == 0).all()) and bool((lse[0] == float("-inf")).all())


def test_long_chunk_over_codes_past_the_largest_half():
    """The code of fp16's largest value stands for 2^16; gathered in fp16 it saturates and the rows stay finite."""
    c = Cache(1, 2, 64, 16, 10, FP, True)
    k, v = _rand((1, 130, 2, 64), FP, 93), _rand((1, 130, 2, 64), FP, 94)
    v[0, 5, 0, 3], v[0, 5, 0, 4], k[0, 5, 0, 9] = 65504, -65504, 65504
    q = _rand((1, 130, 48, 64), FP, 95)
    q[..., 9] = 2.0 ** -14
    A.kv_append(k, v, c.k, c.v, c.table, _i32([130]), **c.scales)
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([130]), **c.scales)
    kk, vv = (np.clip(R.tokens(x, s, c.table_np[0], 130, 16), -65504, 65504) for x, s in ((c.k, c.ks), (c.v, c.vs)))
    assert np.abs(kk).max() == np.abs(vv).max() == 65504
    want = R.attend(R.f64(q[0]), kk, vv, np.arange(130), 0.125, 0, 0)
    R.check_rows(R.f64(o[0]), R.f64(lse[0]), want, R.step(FP), R.step(FP), 64, 130, 65504)


def test_long_chunk_of_a_packed_projection_in_a_graph():
    B, S, Hq, Hkv, D, page = 2, 160, 24, 2, 64, 32
    c = Cache(B, Hkv, D, page, 16, BF, True)
    table, kv = A.rope_table(512, D), _i32([160, 160])
    qkv = _rand((B, S, (Hq + 2 * Hkv) * D), BF, 92)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=-1))

    def step():
        A.kv_append(k, v, c.k, c.v, c.table, kv, table=table, **c.scales)
        return A.attention_paged(q, c.k, c.v, c.table, kv, table=table, **c.scales)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    kv.copy_(_i32([400, 161]))
    for b in range(B):
        c.fill(b, [240, 1][b], 50 + b)
    g.replay()
    torch.cuda.synchronize()
    rot = torch.stack([A.rope_apply(q[b:b + 1].contiguous(), table, pos0=[240, 1][b])[0] for b in range(B)])
    for b in range(B):
        L = [400, 161][b]
        kk, vv = (R.tokens(x, s, c.table_np[b], L, page) for x, s in ((c.k, c.ks), (c.v, c.vs)))
        want = R.attend(R.f64(rot[b]), kk, vv, np.arange(L - S, L), D ** -0.5, 0, 0)
        R.check_rows(R.f64(out[0][b]), R.f64(out[1][b]), want, R.step(BF), R.step(BF), D, L, _v_top(c, c.table_np[b, :13]),
                     f"graph b={b}")


def _scaled_pages(rel_log2, logit_log2, seed):
    """A one-head e4m3 cache of pages whose value scales are 2^rel_log2[j] and whose keys all have logits near
    logit_log2[j] * ln 2 for the query of ones / 64: (cache, query, keys)."""
    D, page = 64, 16
    n = len(rel_log2)
    c = Cache(1, 1, D, page, n, BF, True, seed=seed)
    c.fill(0, n * page, seed)
    q = torch.ones((1, 1, 1, D), dtype=BF, device=DEV)
    for j in range(n):
        at = int(c.table_np[0, j])
        c.vs[at] = 2.0 ** rel_log2[j]
        # K = +-code, D of them alike: q . K scale / 8 = logit
        c.k.view(torch.uint8)[at] = torch.ones((1, page, D), device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
        c.ks[at] = logit_log2[j] * np.log(2.0) / (D * D ** -0.5) if logit_log2[j] else 1e-30
    return c, q, n * page


@pytest.mark.parametrize("rel_log2,logit_log2", [
    ([0, 0, 40, 0], [0, 0, -80, 0]),            # enormous values of no weight
    ([40, 0, 0, 0], [-80, 0, 0, 0]),            # ... met first
    ([30, 0, 0], [0, 60, 90]),                  # large values that later keys outweigh
    ([-100, -100, -100], [0, 1, 0]),            # values of nothing (a block of zeros has this scale)
    ([0, -100, 3], [0, 10, 2]),                 # most of the weight on values of nothing
    ([120, 118, 0], [0, 1, 3]),                 # values near the end of bf16
])
def test_value_scales_far_apart(rel_log2, logit_log2):
    """Each page's contribution counts by weight times scale, scales below 2^-72 as 2^-72. What the 16-bit products lose
    is relative to the largest such contribution: n 2^-24 of 448 max_j p_j max(scale_j, 2^-72) (half a subnormal step,
    2^-25, twice for the sum's side)."""
    c, q, n = _scaled_pages(rel_log2, logit_log2, 5)
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([n]), **c.scales)
    k, v = (R.tokens(x, s, c.table_np[0], n, 16) for x, s in ((c.k, c.ks), (c.v, c.vs)))
    want = R.attend(R.f64(q[0]), k, v, np.array([n - 1]), 64 ** -0.5, 0, 0)
    z = 64 ** -0.5 * k[:, 0].sum(-1)
    w = np.exp(z - z.max())
    w /= w.sum()
    top = float((w * np.repeat(2.0 ** np.maximum(np.array(rel_log2, float), -72), 16)).max() * 448)
    R.check_rows(R.f64(o[0]), R.f64(lse[0]), want, R.step(BF), R.step(FP), 64, n, top, f"{rel_log2} {logit_log2}")


def test_the_native_module_and_the_wrappers_own_checks_agree(monkeypatch):
    """The usual call goes through the native module, others through the wrappers' checks: the same bits, the same
    refusals."""
    class Sub(torch.Tensor):
        pass

    def step(q, k, v, **kw):
        c = Cache(2, 2, 64, 16, 10, BF, True)
        c.fill(0, 130, 0), c.fill(1, 40, 1)
        A.kv_append(k, v, c.k, c.v, c.table, _i32([131, 41]), **c.scales)
        o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([131, 41]), **c.scales, **kw)
        w = A.attention_window(q.repeat(1, 9, 1, 1), k.repeat(1, 9, 1, 1), v.repeat(1, 9, 1, 1), window=3)
        return [c.k.view(torch.uint8), c.ks.view(torch.int32), c.v.view(torch.uint8), c.vs.view(torch.int32), o, lse, *w]

    q, k, v = _rand((2, 1, 8, 64), BF, 1), _rand((2, 1, 2, 64), BF, 2), _rand((2, 1, 2, 64), BF, 3)
    want = step(q, k, v)
    assert A._native is not None
    c = Cache(1, 2, 64, 16, 10, BF, True)
    for native in (A._native, None):
        monkeypatch.setattr(A, "_native", native)
        for got in (step(q, k, v), step(q.as_subclass(Sub), k.as_subclass(Sub), v),
                    step(q, k, v, window=2 ** 40, sinks=2 ** 40, scale=0.125),
                    step(q, k, v, workspace=torch.empty(1 << 22, dtype=torch.uint8, device=DEV)),
                    step(q, k, v, out=torch.empty_like(q), lse=torch.empty(2, 8, 1, device=DEV))):
            for a, b in zip(got, want):
                assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b)
        with pytest.raises(A.AttnError) as e:
            A.attention_paged(q[:1], c.k, c.v, c.table, _i32([3]), **c.scales,
                              workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
        assert e.value.code == A.ATTN_ERR_INVALID_ARG
        with pytest.raises(A.AttnError):
            A.kv_append(k[:1], v[:1], c.k[:, :, :8].contiguous(), c.v[:, :, :8].contiguous(), c.table, _i32([3]), **c.scales)
        with pytest.raises(A.AttnError):
            A.attention_window(q, k, v, window=0)
        for kw in (dict(window=-1), dict(out=torch.empty(1, 1, 8, 64, device=DEV)), dict(q_lens=_i32([1, 1])),
                   dict(k_scale=c.ks[:1]), dict(table=torch.zeros(9, 64, 2, device=DEV)),
                   dict(table=torch.zeros(0, 32, 2, device=DEV))):
            with pytest.raises(ValueError):
                A.attention_paged(q[:1], c.k, c.v, c.table, _i32([3]), **{**c.scales, **kw})
        with pytest.raises(ValueError):
            A.kv_append(k[:1], v, c.k, c.v, c.table, _i32([3]), **c.scales)
        with pytest.raises(ValueError):
            A.attention_window(q, k, v[:, :, :1], window=3)
    assert _status() == A.ATTN_OK


def test_native_calls_of_threads_and_streams_keep_apart():
    """Threads and side streams that call at once, through the native module."""
    import threading
    c = Cache(3, 2, 128, 16, 300, BF, True)
    for b in range(3):
        c.fill(b, [4700, 4000, 1][b], b)
    kv = _i32([4700, 4000, 1])
    qs = [_rand((3, 1, 8, 128), BF, 70 + i) for i in range(4)]
    want = [A.attention_paged(q, c.k, c.v, c.table, kv, **c.scales) for q in qs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream() if i % 2 else torch.cuda.current_stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                o, lse = A.attention_paged(qs[i], c.k, c.v, c.table, kv, **c.scales)
                s.synchronize()
                if not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])):
                    bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [x.start() for x in ts], [x.join() for x in ts]
    assert not bad


@pytest.mark.parametrize("native", [True, False])
def test_empty_problems(native, monkeypatch):
    """No sequence, no token, no page: nothing is launched or written, and shapes come back."""
    c = Cache(2, 2, 64, 16, 3, BF, True)
    c.fill(0, 20, 0), c.fill(1, 5, 1)
    A.attention_paged(_rand((2, 1, 8, 64), BF, 0), c.k, c.v, c.table, _i32([20, 5]), **c.scales)
    if not native:
        monkeypatch.setattr(A, "_native", None)
    was = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks.view(torch.int32))]
    for B, S in ((0, 1), (2, 0), (0, 0)):
        table, lens = c.table[:B].contiguous(), _i32([20, 5][:B])
        k = torch.empty((B, S, 2, 64), dtype=BF, device=DEV)
        A.kv_append(k, k, c.k, c.v, table, lens, **c.scales)
        o, lse = A.attention_paged(torch.empty((B, S, 8, 64), dtype=BF, device=DEV), c.k, c.v, table, lens, **c.scales)
        assert o.shape == (B, S, 8, 64) and lse.shape == (B, 8, S)
        w, wl = A.attention_window(torch.empty((B, S, 8, 64), dtype=BF, device=DEV), k, k, window=4)
        assert w.shape == (B, S, 8, 64) and wl.shape == (B, 8, S)
    with pytest.raises(A.AttnError):
        A.attention_paged(_rand((2, 1, 8, 64), BF, 0), c.k, c.v, c.table[:, :0].contiguous(), _i32([20, 5]), **c.scales)
    o, lse = A.attention_window(_rand((1, 3, 2, 64), BF, 1), *[torch.empty((1, 0, 1, 64), dtype=BF, device=DEV)] * 2, window=2)
    assert bool((o == 0).all()) and bool((lse == float("-inf")).all())
    assert all(torch.equal(a, b) for a, b in zip(was, (c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks.view(torch.int32))))
    assert _status() == A.ATTN_OK


def test_a_windowed_prompt_follows_the_kernel_that_makes_its_inputs():
    """The windowed kernel starts while its producer drains: a chain of producers and windows in a graph and eagerly."""
    B, S, H, D = 2, 700, 8, 128
    x = _rand((B, S, H, D), BF, 5)
    table = A.rope_table(2048, D)

    def chain(x):
        for i in range(6):
            q = A.rope_apply(x, table, pos0=i)
            o, _ = A.attention_window(q, q, x, window=100 + i, sinks=3)
            x = (o + x).contiguous()
        return x

    want = x
    for i in range(6):                                   # the same with a synchronisation at every step
        q = A.rope_apply(want, table, pos0=i)
        torch.cuda.synchronize()
        o, _ = A.attention_window(q, q, want, window=100 + i, sinks=3)
        torch.cuda.synchronize()
        want = (o + want).contiguous()
    assert torch.equal(chain(x), want)
    static = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain(static)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Sq", [(2, 1), (8, 3), (8, 5), (16, 4)])
@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
def test_pages_of_one_tile(e4m3, Hq, Sq, D):
    """Pages of 16 tokens: every tile of a stage has a page and scales of its own, some out of range (their keys are
    hidden), some wholly before the window, the last one ragged."""
    Hkv, page, n = 2 if Hq < 16 else 1, 16, 16 * 70 + 5
    c = Cache(1, Hkv, D, page, 72, BF, e4m3, seed=D + Hq)
    c.fill(0, n, 3)
    if e4m3:
        for j in range(0, 71, 3):
            c.vs[int(c.table_np[0, j])] *= 2.0 ** (j % 7)
    gone = [5, 6, 17, 40, 63]
    table = c.table.clone()
    for i, j in enumerate(gone):
        table[0, j] = [-1, 1 << 30, -(1 << 31), 74 + 0, 1000][i]
    q = _rand((1, Sq, Hq, D), BF, 7)
    keep = np.array([t // page not in gone for t in range(n)])
    for window, sinks in ((0, 0), (600, 70), (33, 0)):
        o, lse = A.attention_paged(q, c.k, c.v, table, _i32([n]), window=window, sinks=sinks, **c.scales)
        bad = _status()
        k, v = (R.tokens(x, s, c.table_np[0], n, page) for x, s in ((c.k, c.ks), (c.v, c.vs)))
        pos = np.arange(n - Sq, n)
        for i in range(Sq):
            t = np.arange(n)
            see = keep & (t <= pos[i]) & (True if not window else (t > pos[i] - window) | (t < sinks))
            ks, vs = k[see], v[see]
            want = R.attend(R.f64(q[0, i:i + 1]), ks, vs, np.array([len(ks) - 1]), D ** -0.5, 0, 0)
            R.check_rows(R.f64(o[0, i:i + 1]), R.f64(lse[0, :, i:i + 1]), want, R.step(BF),
                         R.step(FP) if e4m3 else R.step(BF), D, n, _v_top(c, c.table_np[0, :71]), f"{window} {i}")
        assert bad == (A.ATTN_OK if window == 33 else A.ATTN_ERR_BAD_INDEX)


@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "16bit"])
@pytest.mark.parametrize("Hq,Hkv,D,Sq", [(8, 2, 128, 1), (8, 8, 64, 1), (7, 1, 128, 5), (16, 2, 64, 3), (12, 2, 128, 20)])
def test_short_tables(Hq, Hkv, D, Sq, e4m3):
    """Tables that a CTA takes whole (256 keys): empty sequences, no queries, more queries than keys, lengths out of
    range; and the same lengths under a table that goes by the schedule."""
    kv, ql = [256, 0, 17, 1, 200, 130, 5], [Sq, Sq, max(Sq - 1, 0), Sq, 0, Sq, Sq]
    B, page = len(kv), 32
    c = Cache(B, Hkv, D, page, 8, FP, e4m3, seed=Hq * D)
    for b in range(B):
        c.fill(b, kv[b], b)
    q = _rand((B, Sq, Hq, D), FP, 8)
    wide = torch.cat([c.table, torch.full((B, 100), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    for window, sinks in ((0, 0), (20, 3)):
        for table in (c.table, wide):
            o, lse = torch.full_like(q, 5.0), torch.full((B, Hq, Sq), 5.0, device=DEV)
            A.attention_paged(q, c.k, c.v, table, _i32(kv), q_lens=_i32(ql), window=window, sinks=sinks, out=o, lse=lse,
                              **c.scales)
            assert _status() == A.ATTN_OK
            _check_attention(c, q, q, o, lse, kv, ql, window, sinks, label=f"{window} {table.shape}")
            for b in range(B):
                assert bool((o[b, ql[b]:] == 5.0).all()) and bool((lse[b, :, ql[b]:] == 5.0).all())
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([-1, 300, 17, 1, 200, 130, 5]), **c.scales)
    assert _status() == A.ATTN_ERR_BAD_INDEX
    assert bool((o[0] == 0).all()) and bool((lse[0] == float("-inf")).all()) and bool(torch.isfinite(o[2:]).all())
