"""Cases of the serving operators: appending to a paged key/value cache, attention over it, windowed prefill.

Three operators, each a case's ``op``:

* ``append``: new keys and values of B sequences enter a paged cache, the keys rotated to their positions; an 8-bit
  (e4m3) cache holds one power-of-two scale for each page and head, which grows with the page's values.
* ``paged``: attention of the step's queries over such a cache, optionally with a sliding window and sinks.
* ``window``: causal attention on contiguous tensors with a sliding window and sinks (prefill).

Lengths of ragged batches depend on the case alone, values on the seed.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -100           # the smallest block scale is 2**MIN_EXP
BASE = 10000.0           # rotary base


# ------------------------------------------------------------------- cases

def _append(name, B, S, Hkv, D, page, ctx, dtype, cache, rope=True, ragged=False):
    return dict(name=name, op="append", B=B, S=S, Hkv=Hkv, D=D, page=page, ctx=ctx, dtype=dtype, cache=cache,
                rope=rope, ragged=ragged)


def _paged(name, B, Sq, Hq, Hkv, D, page, ctx, dtype, cache, window=0, sinks=0, rope=True, ragged=False):
    return dict(name=name, op="paged", B=B, Sq=Sq, Hq=Hq, Hkv=Hkv, D=D, page=page, ctx=ctx, dtype=dtype, cache=cache,
                window=window, sinks=sinks, rope=rope, ragged=ragged)


def _window(name, B, Hq, Hkv, Sq, Sk, D, window, sinks, dtype):
    return dict(name=name, op="window", B=B, Hq=Hq, Hkv=Hkv, Sq=Sq, Sk=Sk, D=D, window=window, sinks=sinks,
                dtype=dtype)


def listed():
    return [
        # one sequence's decode step: latency is all there is
        _append("append_one_token", 1, 1, 8, 128, 64, 4096, "bf16", "e4m3"),
        # a decode step of a ragged batch (one slot of it idle), GQA heads
        _append("append_decode_batch", 64, 1, 8, 128, 64, 8192, "bf16", "e4m3", ragged=True),
        # the prompts of the Llama-2-7B-shaped prefill enter an 8-bit cache, on top of a short common prefix
        _append("append_prefill_e4m3", 4, 2048, 32, 128, 64, 37, "bf16", "e4m3"),
        # chunked prefill of a ragged batch into a 16-bit cache, head size 64
        _append("append_chunk_f16", 8, 500, 8, 64, 16, 1000, "f16", "16bit", ragged=True),
        # one short conversation's decode step
        _paged("paged_one_short", 1, 1, 32, 8, 128, 64, 500, "bf16", "e4m3"),
        # the GQA decode workload of the benchmark (16 sequences of 8192 keys) over the 8-bit cache
        _paged("paged_gqa_decode", 16, 1, 32, 8, 128, 64, 8192, "bf16", "e4m3"),
        # long contexts, few sequences: the key axis has to be split
        _paged("paged_long_decode", 4, 1, 32, 8, 128, 64, 32768, "bf16", "e4m3", ragged=True),
        # multi-head decode over a 16-bit cache, the benchmark's MHA decode lengths, small pages
        _paged("paged_mha_16bit", 16, 1, 32, 32, 128, 16, 4096, "f16", "16bit"),
        # several draft tokens a sequence, windowed with sinks, ragged
        _paged("paged_draft_window", 32, 5, 32, 8, 64, 32, 12000, "bf16", "e4m3", window=4096, sinks=4, ragged=True),
        # a short windowed prompt of odd length
        _window("window_short", 1, 32, 8, 777, 777, 128, 256, 4, "bf16"),
        # the Llama-2-7B-shaped prefill at head size 64 with a narrow window, fp16
        _window("window_narrow_d64", 4, 32, 32, 2048, 2048, 64, 512, 0, "f16"),
        # a long GQA prompt with the usual 4096-token window and sinks
        _window("window_long_gqa", 1, 32, 8, 16384, 16384, 128, 4096, 4, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "window"])
    D, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice(["e4m3", "e4m3", "16bit"])
    page = rng.choice([16, 32, 64, 128])
    while True:
        if op == "append":
            B, S = _log(rng, 1, 64), rng.choice([1, _log(rng, 2, 2048)])
            Hkv, ctx = rng.choice([1, 2, 4, 8, 8, 16, 32]), _log(rng, 1, 8192)
            if B * S * Hkv * D <= 1 << 25 and B * (S + ctx) * Hkv * D <= 1 << 28:
                c = _append("", B, S, Hkv, D, page, ctx, dtype, cache, rng.random() < 0.8, rng.random() < 0.5)
                break
        elif op == "paged":
            B, Sq = _log(rng, 1, 64), rng.choice([1, 1, rng.randint(2, 8)])
            Hkv, G, ctx = rng.choice([1, 2, 4, 8, 8, 32]), rng.choice([1, 2, 3, 4, 4, 7, 8]), _log(rng, 1, 32768)
            if Hkv * G <= 64 and B * ctx * Hkv * D * (1 if cache == "e4m3" else 2) <= 1 << 27 and \
                    B * ctx * Hkv * G * Sq <= 1 << 27:
                window = rng.choice([0, 0, _log(rng, 1, ctx)])
                c = _paged("", B, Sq, Hkv * G, Hkv, D, page, max(ctx, Sq), dtype, cache, window,
                           rng.choice([0, 4, 19]) if window else 0, rng.random() < 0.8, rng.random() < 0.5)
                break
        else:
            B, Hkv, G = rng.choice([1, 1, 2, 4]), rng.choice([1, 2, 4, 8, 32]), rng.choice([1, 2, 4, 4, 7, 8])
            Sk = _log(rng, 16, 16384)
            Sq = rng.choice([Sk, Sk, Sk, rng.randint(1, Sk)])
            if Hkv * G <= 64 and B * Hkv * G * Sq * Sk <= 1 << 32:
                c = _window("", B, Hkv * G, Hkv, Sq, Sk, D, _log(rng, 1, Sk), rng.choice([0, 4, 4, 130]), dtype)
                break
    del c["name"]
    return c


# ---------------------------------------------------- lengths and positions

def _lens(case):
    """(kv_lens, new_lens) as lists: tokens in the cache including the step's, tokens of the step."""
    B, S = case["B"], case["S"] if case["op"] == "append" else case["Sq"]
    ctx = case["ctx"] + (S if case["op"] == "append" else 0)
    if not case["ragged"]:
        return [ctx] * B, [S] * B
    kv, new = [], []
    for b in range(B):
        if B >= 4 and b == 1:                      # an idle slot of a padded batch
            kv.append(0)
            new.append(0)
            continue
        part = ((5 * b + B // 2) % B) / B
        n = max(1, S - int(part * S / 2))
        new.append(n)
        kv.append(max(n, ctx - int(part * ctx * 0.75)))
    return kv, new


def _visible(case, kv_len, new):
    """(keys that any query of the sequence sees, visible (query, key) pairs)."""
    if new == 0 or kv_len == 0:
        return 0, 0
    W, sinks = case["window"], case["sinks"]
    pos = torch.arange(kv_len - new, kv_len, dtype=torch.int64)
    pos = pos[pos >= 0]
    if W == 0:
        return kv_len, int((pos + 1).sum())
    pairs = int((torch.clamp(pos + 1, max=W) + torch.clamp(torch.clamp(pos + 1 - W, min=0), max=sinks)).sum())
    low = max(0, int(pos[0]) + 1 - W)
    return kv_len - low + min(sinks, low), pairs


def work(case):
    if case["op"] == "window":
        el, B, D = 2, case["B"], case["D"]
        keys, pairs = _visible(case, case["Sk"], case["Sq"])
        return {"bytes": B * (2 * case["Sq"] * case["Hq"] * D * el + 2 * keys * case["Hkv"] * D * el
                              + 4 * case["Hq"] * case["Sq"]),
                "flops": 4.0 * B * case["Hq"] * D * pairs}
    kv, new = _lens(case)
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    ce = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        T = sum(new)
        blocks = sum((k - 1) // page - (k - n) // page + 1 for k, n in zip(kv, new) if n)
        return {"bytes": 2 * T * Hkv * D * (2 + ce) + (T * D * 4 if case["rope"] else 0) + 4 * (blocks + 2 * len(kv))
                + (2 * 4 * blocks * Hkv if ce == 1 else 0), "flops": 5.0 * T * Hkv * D}
    T, total, pages, pairs = sum(new), 0, 0, 0
    for k, n in zip(kv, new):
        keys, p = _visible(case, k, n)
        total, pairs, pages = total + keys, pairs + p, pages + -(-keys // page)
    return {"bytes": 2 * total * Hkv * D * ce + (8 * pages * Hkv if ce == 1 else 0) + 4 * pages
            + T * case["Hq"] * (D * 4 + 4), "flops": 4.0 * case["Hq"] * D * pairs}


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _angles(max_pos, D, dev):
    """(max_pos, D/2, 2) FP32 {cos, sin} of pos * BASE^(-2i/D)."""
    theta = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * torch.pow(
        torch.tensor(BASE, dtype=torch.float64, device=dev),
        torch.arange(D // 2, dtype=torch.float64, device=dev) * (-2.0 / D))
    return torch.stack([theta.cos(), theta.sin()], dim=-1).float().contiguous()


def _block_scale(a):
    """The smallest power of two s with a <= 448 s (at least 2^MIN_EXP), as FP32."""
    m, e = torch.frexp(a)                               # a = m 2^e, 1/2 <= m < 1
    e = torch.where(m > 0.875, e - 8, e - 9)            # 448 = 0.875 * 2^9
    e = torch.where(a > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(a, dtype=torch.float32), e)


def _pages(cache, ids):
    """cache[ids]; 8-bit values are moved as bytes."""
    return cache[ids] if cache.element_size() > 1 else cache.view(torch.uint8)[ids].view(cache.dtype)


def _cache(shape, kind, dt, dev, g):
    """A filled cache of `shape` (pages, heads, page, D) and its scales (None for 16 bits): magnitudes differ by page."""
    x = torch.empty(shape, dtype=dt, device=dev).normal_(generator=g)
    x.mul_(torch.empty((shape[0], shape[1], 1, 1), device=dev).uniform_(0.5, 2.0, generator=g).to(dt))
    if kind == "16bit":
        return x, None
    s = _block_scale(x.abs().amax(dim=(2, 3)).float())
    q = (x.float() / s[:, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, s


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _dtype(case)
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device=dev).normal_(generator=g)

    s = dict(case=case)
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "window":
        s.update(q=normal(case["B"], case["Sq"], case["Hq"], D), k=normal(case["B"], case["Sk"], Hkv, D),
                 v=normal(case["B"], case["Sk"], Hkv, D))
        return s
    B, page = case["B"], case["page"]
    kv, new = _lens(case)
    S = case["S"] if case["op"] == "append" else case["Sq"]
    max_pages = -(-max(kv) // page) + 1                  # room for the next tokens
    n_pages = B * max_pages + 3
    s["k_cache"], s["k_scale"] = _cache((n_pages, Hkv, page, D), case["cache"], dt, dev, g)
    s["v_cache"], s["v_scale"] = _cache((n_pages, Hkv, page, D), case["cache"], dt, dev, g)
    s["block_table"] = torch.randperm(n_pages, device=dev, generator=g)[:B * max_pages].reshape(B, max_pages).int()
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["new_lens"] = torch.tensor(new, dtype=torch.int32, device=dev) if case["ragged"] else None
    s["table"] = _angles(max_pages * page, D, dev) if case["rope"] else None
    if case["op"] == "append":
        s.update(k=normal(B, S, Hkv, D), v=normal(B, S, Hkv, D))
    else:
        # the outputs a serving loop keeps; rows behind a sequence's last query stay as they are
        s.update(q=normal(B, S, case["Hq"], D), out=torch.zeros((B, S, case["Hq"], D), dtype=dt, device=dev),
                 lse=torch.full((B, case["Hq"], S), float("-inf"), device=dev))
    return s


# ------------------------------------------------------------- plain forms

def _rotate(x, table, pos):
    """x (B, S, H, D) in FP32 with row (b, s) at position pos[b, s]."""
    a = table[pos.clamp(min=0)][:, :, None]                            # (B, S, 1, D/2, 2)
    x0, x1, c, n = x[..., 0::2], x[..., 1::2], a[..., 0], a[..., 1]
    return torch.stack([x0 * c - x1 * n, x1 * c + x0 * n], dim=-1).flatten(-2)


def _soft_rows(scores, hidden, v):
    """softmax(scores) v and the row log-sum-exp; scores (FP32) is overwritten. Rows all hidden give 0 and -inf."""
    scores.masked_fill_(hidden, float("-inf"))
    m = scores.amax(dim=-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    scores.sub_(m).exp_()
    total = scores.sum(dim=-1, keepdim=True)
    o = torch.matmul(scores, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (m + total.log()).squeeze(-1)


def _hidden(pos, keys, window, sinks):
    """True where key j is hidden from the query at pos (any leading shape); window 0: the whole past is visible."""
    j = torch.arange(keys, device=pos.device)
    p = pos[..., None]
    h = j > p
    if window:
        h = h | ((j <= p - window) & (j >= sinks))
    return h


def _plain_window(s):
    case, q, k, v = s["case"], s["q"], s["k"], s["v"]
    B, Sq, Hq, D = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    qf = q.float().reshape(B, Sq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)      # (B, Hkv, G, Sq, D)
    kf, vf = (t.float().permute(0, 2, 1, 3)[:, :, None] for t in (k, v))         # (B, Hkv, 1, Sk, D)
    scores = torch.matmul(qf * (1.0 / math.sqrt(D)), kf.transpose(-1, -2))
    pos = torch.arange(Sq, device=q.device) + (Sk - Sq)
    o, lse = _soft_rows(scores, _hidden(pos, Sk, case["window"], case["sinks"]), vf)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, D).to(q.dtype), lse.reshape(B, Hq, Sq)


def _steps(s, S):
    """Per sequence: tokens of the step, and the position of each of its S rows."""
    kv = s["kv_lens"].long()
    new = torch.full_like(kv, S) if s["new_lens"] is None else s["new_lens"].long()
    return kv, new, (kv - new)[:, None] + torch.arange(S, device=kv.device)


def _plain_paged(s):
    case, q = s["case"], s["q"]
    B, Sq, Hq, D = q.shape
    Hkv, G = case["Hkv"], Hq // case["Hkv"]
    kv, new, pos = _steps(s, Sq)
    pages = s["block_table"].long()

    def dense(cache, scale):                                            # (B, Hkv, keys, D) FP32
        x = _pages(cache, pages).float()
        if scale is not None:
            x = x * scale[pages][..., None, None]
        return x.permute(0, 2, 1, 3, 4).flatten(2, 3)

    qf = q.float()
    if s["table"] is not None:
        qf = _rotate(qf, s["table"], pos).to(q.dtype).float()           # the rotated queries are 16-bit values
    qf = (qf * (1.0 / math.sqrt(D))).reshape(B, Sq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Sq, D)
    scores = torch.matmul(qf, dense(s["k_cache"], s["k_scale"]).transpose(-1, -2))
    keys = scores.shape[-1]
    hide = _hidden(pos, keys, case["window"], case["sinks"])[:, None, None]               # (B, 1, 1, Sq, keys)
    vf = dense(s["v_cache"], s["v_scale"])
    o, lse = _soft_rows(scores.reshape(B, Hkv, G, Sq, keys), hide, vf[:, :, None])
    there = (torch.arange(Sq, device=q.device) < new[:, None])
    o = torch.where(there[:, :, None, None], o.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, D).to(q.dtype), s["out"])
    lse = torch.where(there[:, None], lse.reshape(B, Hq, Sq), s["lse"])
    return o, lse


def _plain_append(s):
    case, page = s["case"], s["case"]["page"]
    B, S, Hkv, D = s["k"].shape
    kv, new, pos = _steps(s, S)
    first = kv - new
    # The pages the step touches, at most n of them a sequence; a sequence with fewer repeats its last one, which
    # is then written again with the same values (an idle sequence writes back what it read).
    n = (S + page - 2) // page + 1
    at = torch.minimum(first[:, None] // page + torch.arange(n, device=kv.device),
                       ((kv - 1).clamp(min=0) // page)[:, None])
    ids = torch.gather(s["block_table"].long(), 1, at)                                    # (B, n)
    slot_pos = at[:, :, None] * page + torch.arange(page, device=kv.device)               # (B, n, page)
    is_new = (slot_pos >= first[:, None, None]) & (slot_pos < kv[:, None, None])
    is_old = slot_pos < first[:, None, None]
    row = (slot_pos - first[:, None, None]).clamp(0, S - 1).flatten(1)                    # source row of each slot
    old_page = is_old.any(-1)[:, :, None]                                                 # (B, n, 1)

    def put(x, cache, scale):
        got = torch.gather(x, 1, row[:, :, None, None].expand(-1, -1, Hkv, D))
        got = got.reshape(B, n, page, Hkv, D).permute(0, 1, 3, 2, 4)                      # (B, n, Hkv, page, D)
        m_new, m_old = is_new[:, :, None, :, None], is_old[:, :, None, :, None]
        have = _pages(cache, ids)
        if scale is None:
            cache[ids] = torch.where(m_new, got.to(cache.dtype), have)
            return
        need = _block_scale((got.abs() * m_new).amax(dim=(3, 4)))
        before = scale[ids]
        grown = torch.where(is_new.any(-1)[:, :, None], torch.where(old_page, torch.maximum(before, need), need), before)
        codes = (got / grown[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX)
        moved = have.float() * (before / grown)[..., None, None]
        kept = torch.where(m_old, moved, have.float())
        cache.view(torch.uint8)[ids] = torch.where(m_new, codes, kept).to(cache.dtype).view(torch.uint8)
        scale[ids] = grown

    kf = s["k"].float()
    if s["table"] is not None:
        kf = _rotate(kf, s["table"], pos.clamp(max=s["table"].shape[0] - 1))
    put(kf, s["k_cache"], s["k_scale"])
    put(s["v"].float(), s["v_cache"], s["v_scale"])
    return _caches(s)


def _caches(s):
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if s[n] is not None}


def run(s):
    case = s["case"]
    if not own:
        return {"append": _plain_append, "paged": _plain_paged, "window": _plain_window}[case["op"]](s)
    import transformer_attention_02_gb300 as ta
    if case["op"] == "window":
        return ta.attention_window(s["q"], s["k"], s["v"], window=case["window"], sinks=case["sinks"])
    if case["op"] == "append":
        ta.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                     new_lens=s["new_lens"], k_scale=s["k_scale"], v_scale=s["v_scale"], table=s["table"])
        return _caches(s)
    return ta.attention_paged(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                              q_lens=s["new_lens"], k_scale=s["k_scale"], v_scale=s["v_scale"], table=s["table"],
                              window=case["window"], sinks=case["sinks"], out=s["out"], lse=s["lse"])


# ------------------------------------------------------ the values in 64 bits

def _turn64(x, table, pos):
    """One row set x (rows, H, D) in FP64 turned by the table's angles at pos (rows)."""
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], -1, 2).contiguous())
    w = torch.view_as_complex(table.double()[pos].contiguous())[:, None]
    return torch.view_as_real(z * w).reshape(x.shape)


def _attend64(q, k, v, pos, key_pos, window, sinks):
    """q (R, H, D) at pos (R), k and v (L, H, D) at key_pos (L), all FP64: o (R, H, D), lse (H, R)."""
    z = torch.einsum("rhd,lhd->hrl", q, k) / math.sqrt(q.shape[-1])
    dist = pos[:, None] - key_pos[None]
    see = dist >= 0
    if window:
        see &= (dist < window) | (key_pos < sinks)[None]
    z = torch.where(see, z, torch.tensor(float("-inf"), dtype=z.dtype, device=z.device))
    lse = torch.logsumexp(z, dim=-1)
    w = torch.where(see, (z - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None]).exp(),
                    torch.zeros((), dtype=z.dtype, device=z.device))
    return torch.einsum("hrl,lhd->rhd", w, v), lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "window":
        return _exact_window(case, s)
    if case["op"] == "paged":
        return _exact_paged(case, s)
    return _exact_append(case, s)


def _exact_window(case, s):
    q, k, v = s["q"], s["k"], s["v"]
    B, Sq, Hq, D = q.shape
    Sk, G = k.shape[1], Hq // k.shape[2]
    o = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty((B, Hq, Sq), dtype=torch.float64, device=q.device)
    for b in range(B):
        for i0 in range(0, Sq, 1024):
            i1 = min(Sq, i0 + 1024)
            pos = torch.arange(i0, i1, device=q.device) + (Sk - Sq)
            lo = max(0, i0 + Sk - Sq + 1 - case["window"])
            hi = max(0, i1 + Sk - Sq)
            keys = torch.arange(hi, device=q.device)
            keys = keys[(keys >= lo) | (keys < case["sinks"])]
            kk, vv = (t[b, keys].double().repeat_interleave(G, dim=1) for t in (k, v))
            o[b, i0:i1], lse[b, :, i0:i1] = _attend64(q[b, i0:i1].double(), kk, vv, pos, keys, case["window"],
                                                     case["sinks"])
    return o, lse


def _exact_paged(case, s):
    q, page, D = s["q"], case["page"], case["D"]
    G = case["Hq"] // case["Hkv"]
    kv, new = _lens(case)
    o, lse = s["out"].double(), s["lse"].double()
    for b, (L, n) in enumerate(zip(kv, new)):
        if n == 0 or L == 0:
            continue
        ids = s["block_table"][b, :-(-L // page)].long()

        def tokens(cache, scale):
            x = _pages(cache, ids).double()
            if scale is not None:
                x = x * scale[ids].double()[:, :, None, None]
            return x.transpose(1, 2).reshape(-1, case["Hkv"], D)[:L].repeat_interleave(G, dim=1)

        pos = torch.arange(L - n, L, device=q.device)
        qb = q[b, :n].double()
        if s["table"] is not None:
            qb = _turn64(q[b, :n], s["table"], pos).to(q.dtype).double()
        o[b, :n], lse[b, :, :n] = _attend64(qb, tokens(s["k_cache"], s["k_scale"]), tokens(s["v_cache"], s["v_scale"]),
                                            pos, torch.arange(L, device=q.device), case["window"], case["sinks"])
    return o, lse


def _exact_append(case, s):
    page, dev = case["page"], s["k"].device
    kv, new = _lens(case)
    got = {n: t.double() for n, t in _caches(s).items()}
    for b, (L, n) in enumerate(zip(kv, new)):
        if n == 0:
            continue
        pos = torch.arange(L - n, L, device=dev)
        kb = s["k"][b, :n].double() if s["table"] is None else _turn64(s["k"][b, :n], s["table"], pos)
        for which, x in (("k", kb), ("v", s["v"][b, :n].double())):
            cache, scale = got[which + "_cache"], got.get(which + "_scale")
            ids = s["block_table"][b].long()[pos // page]
            if scale is not None:
                touched = torch.unique_consecutive(ids)
                first = (L - n) % page                        # slots of the first page that were filled before
                group = pos // page - (L - n) // page
                top = torch.zeros((len(touched), case["Hkv"]), dtype=torch.float64, device=dev)
                top.scatter_reduce_(0, group[:, None].expand(-1, case["Hkv"]), x.abs().amax(-1), "amax")
                e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 2.0 ** -120)) / E4M3_MAX))
                fresh = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=dev), e.clamp(min=MIN_EXP))
                if first:
                    was = scale[touched[0]].clone()
                    fresh[0] = torch.maximum(fresh[0], was)
                    cache[touched[0], :, :first] *= (was / fresh[0])[:, None, None]
                scale[touched] = fresh
                x = x / fresh[group][..., None]
            cache[ids, :, pos % page] = x
    return got
