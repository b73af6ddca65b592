"""Cases of the training operators: attention's backward pass, rotary positions with several axes, 8-bit checkpoints.

Four operators, each a case's ``op``:

* ``backward``: the gradients of Q, K and V of an attention (causal, windowed with sinks, additively masked, or over all
  keys) from the gradient of its output, its output and its row log-sum-exp; the probabilities are recomputed.
* ``rope``: queries and keys turned by positions of several axes (time, height, width), or turned back (the gradient).
* ``store``: an activation (B, S, H, D) kept in 8 bits: e4m3 codes and a power of two for each head vector.
* ``from8``: the same gradients from 8-bit checkpoints of Q, K and V alone; the output is computed again.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -100           # the smallest scale is 2**MIN_EXP
BASE = 10000.0           # rotary base


# ------------------------------------------------------------------- cases

def _backward(name, B, Hq, Hkv, Sq, Sk, D, dtype, causal=True, window=0, sinks=0, masked=False, packed=False):
    return dict(name=name, op="backward", B=B, Hq=Hq, Hkv=Hkv, Sq=Sq, Sk=Sk, D=D, dtype=dtype, causal=causal, window=window,
                sinks=sinks, masked=masked, packed=packed)


def _rope(name, B, S, Hq, Hkv, sections, grid, dtype, own_freqs=False, inverse=False, packed=False):
    """sections: rotated pairs of time, height and width, as one text; grid: patches of a picture's row (0: text)."""
    return dict(name=name, op="rope", B=B, S=S, Hq=Hq, Hkv=Hkv, sections=sections, grid=grid, dtype=dtype,
                own_freqs=own_freqs, inverse=inverse, packed=packed)


def _store(name, B, S, H, D, dtype, packed=False):
    return dict(name=name, op="store", B=B, S=S, H=H, D=D, dtype=dtype, packed=packed)


def _from8(name, B, Hq, Hkv, S, D, dtype, window=0, sinks=0):
    return dict(name=name, op="from8", B=B, Hq=Hq, Hkv=Hkv, Sq=S, Sk=S, D=D, dtype=dtype, causal=True, window=window,
                sinks=sinks, masked=False)


def listed():
    return [
        # one short sample: latency is all there is
        _backward("backward_short", 1, 8, 2, 100, 100, 64, "bf16"),
        # a training step of the benchmark's Llama-2-7B-shaped layer
        _backward("backward_llama2_7b", 4, 32, 32, 2048, 2048, 128, "bf16"),
        # the benchmark's GQA workload, gradients of shared heads, Q, K and V inside a packed projection
        _backward("backward_gqa", 8, 32, 8, 4096, 4096, 128, "bf16", packed=True),
        # cross attention of odd lengths, fp16, head size 64
        _backward("backward_cross_f16", 3, 16, 16, 777, 1301, 64, "f16", causal=False),
        # a long windowed sample with sinks
        _backward("backward_window_long", 1, 32, 8, 16384, 16384, 128, "bf16", window=4096, sinks=4),
        # an additive mask that hides three keys of ten and some rows whole (the stress workloads' sizes)
        _backward("backward_masked", 2, 16, 16, 2048, 2048, 128, "bf16", causal=False, masked=True),
        # a decode step's tokens of a ragged position each
        _rope("rope_decode", 32, 1, 32, 8, "16,24,24", 0, "bf16"),
        # prompts with pictures: text and patches in one sequence, Q and K inside a packed projection
        _rope("rope_pictures", 4, 4097, 32, 8, "16,24,24", 64, "bf16", packed=True),
        # the gradient's way back through a video's positions, fp16, head size 64, each axis with frequencies of its own
        _rope("rope_video_back", 1, 33000, 24, 24, "8,12,12", 52, "f16", own_freqs=True, inverse=True),
        # a short sample's keys
        _store("store_small", 1, 333, 8, 64, "f16"),
        # the values of the Llama-2-7B-shaped layer, out of a packed projection
        _store("store_llama2_7b", 4, 2048, 32, 128, "bf16", packed=True),
        # a layer's backward pass from 8-bit checkpoints
        _from8("from8_gqa", 2, 32, 8, 4096, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["backward", "backward", "backward", "rope", "store", "from8"])
    D, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "f16"])
    while True:
        if op == "backward":
            B, Hkv, G = _log(rng, 1, 8), rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 1, 2, 3, 4, 7, 8])
            Sk = _log(rng, 1, 16384)
            Sq = rng.choice([Sk, Sk, Sk, _log(rng, 1, 16384)])
            kind = rng.choice(["all", "causal", "causal", "window", "masked"])
            if Hkv * G > 64 or B * Hkv * G * Sq * Sk > 1 << 32 or (kind == "masked" and B * Sq * Sk > 1 << 28):
                continue
            c = _backward("", B, Hkv * G, Hkv, Sq, Sk, D, dtype, kind in ("causal", "window"),
                          _log(rng, 1, Sk) if kind == "window" else 0, rng.choice([0, 4, 130]) if kind == "window" else 0,
                          kind == "masked", Sq == Sk and rng.random() < 0.5)
        elif op == "rope":
            B, S = _log(rng, 1, 32), rng.choice([1, _log(rng, 2, 33000)])
            Hkv, G = rng.choice([1, 2, 4, 8, 24]), rng.choice([1, 2, 4, 5])
            if Hkv * G > 64 or B * S * Hkv * (G + 1) * D > 1 << 27:
                continue
            n = D // 2
            t = rng.randint(1, n - 2)
            h = rng.randint(1, n - t - 1)
            sections = rng.choice(["16,24,24" if D == 128 else "8,12,12", f"{t},{h},{n - t - h}", f"{t},{n - t}", f"{n}"])
            c = _rope("", B, S, Hkv * G, Hkv, sections, rng.choice([0, 7, 64]), dtype, rng.random() < 0.5,
                      rng.random() < 0.4, rng.random() < 0.5)
        elif op == "store":
            B, S, H = _log(rng, 1, 8), _log(rng, 1, 16384), rng.choice([1, 2, 8, 24, 32])
            if B * S * H * D > 1 << 27:
                continue
            c = _store("", B, S, H, D, dtype, rng.random() < 0.5)
        else:
            B, Hkv, G, S = _log(rng, 1, 4), rng.choice([1, 2, 8, 16]), rng.choice([1, 2, 4]), _log(rng, 1, 8192)
            if B * Hkv * G * S * S > 1 << 31:
                continue
            window = rng.choice([0, 0, _log(rng, 1, S)])
            c = _from8("", B, Hkv * G, Hkv, S, D, dtype, window, 4 if window else 0)
        del c["name"]
        return c


# ------------------------------------------------------------------- sizes

def _visible(case):
    """(visible (query, key) pairs of one head, keys that any query sees, queries that see any key), a mask aside."""
    Sq, Sk, W, sinks = case["Sq"], case["Sk"], case["window"], case["sinks"]
    if not case["causal"]:
        return Sq * Sk, (Sk if Sq else 0), (Sq if Sk else 0)
    pos = torch.arange(Sq, dtype=torch.int64) + (Sk - Sq)
    pos = pos[pos >= 0]
    if len(pos) == 0:
        return 0, 0, 0
    if not W:
        return int((pos + 1).sum()), Sk, len(pos)
    pairs = int((torch.clamp(pos + 1, max=W) + torch.clamp(torch.clamp(pos + 1 - W, min=0), max=sinks)).sum())
    low = max(0, int(pos[0]) + 1 - W)
    return pairs, Sk - low + min(sinks, low), len(pos)


def work(case):
    B, D = case["B"], _head(case)
    if case["op"] == "rope":
        n = B * case["S"] * (case["Hq"] + case["Hkv"]) * D
        axes = len(case["sections"].split(","))
        return {"bytes": 4 * n + 4 * B * case["S"] * axes, "flops": 3.0 * n}
    if case["op"] == "store":
        n = B * case["S"] * case["H"] * D
        return {"bytes": 3 * n + 4 * n // D, "flops": 2.0 * n}
    Hq, Hkv, Sq, Sk = case["Hq"], case["Hkv"], case["Sq"], case["Sk"]
    pairs, keys, _ = _visible(case)
    if case["masked"]:
        pairs = B * Sq * (Sk - int(0.3 * Sk)) // B              # three keys of ten are hidden
    nq, nk = B * Sq * Hq * D, B * keys * Hkv * D
    if case["op"] == "from8":                                    # codes and scales in, dO in, three gradients out
        b = (nq + 2 * nk) * (1 + 4 / D) + 2 * nq + 2 * nq + 2 * 2 * B * Sk * Hkv * D
        return {"bytes": int(b), "flops": 14.0 * B * Hq * D * pairs}
    b = 2 * (3 * nq + 2 * nk) + 4 * B * Sq * Hq + 2 * nq + 2 * 2 * B * Sk * Hkv * D
    return {"bytes": b + (4 * B * Sq * Sk if case["masked"] else 0), "flops": 10.0 * B * Hq * D * pairs}


def _head(case):
    return 2 * sum(int(n) for n in case["sections"].split(",")) if case["op"] == "rope" else case["D"]


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _sections(case):
    return [int(n) for n in case["sections"].split(",")]


def _angles(max_pos, sections, own_freqs, dev):
    """(max_pos, D/2, 2) FP32 {cos, sin}: of pos * BASE^(-2i/D), or, each axis with its own frequencies, BASE^(-j/n)."""
    if own_freqs:
        e = torch.cat([torch.arange(n, dtype=torch.float64) / n for n in sections])
    else:
        e = torch.arange(sum(sections), dtype=torch.float64) / sum(sections)
    theta = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * torch.pow(
        torch.tensor(BASE, dtype=torch.float64), -e).to(dev)
    return torch.stack([theta.cos(), theta.sin()], dim=-1).float().contiguous()


def _positions(case, dev, g):
    """(B, S, axes) int32. A decode step's tokens sit anywhere; a sequence runs through text, where all axes count alike,
    and then row by row through pictures (or a video's frames)."""
    B, S, axes, w = case["B"], case["S"], len(_sections(case)), case["grid"]
    if S == 1:
        at = torch.randint(0, 8192, (B, 1, 1), device=dev, generator=g)
        return at.expand(B, S, axes).contiguous().int()
    s = torch.arange(S, device=dev)
    if not w:
        return s[None, :, None].expand(B, S, axes).contiguous().int()
    text = torch.randint(0, min(S, 64), (B, 1), device=dev, generator=g)
    p = (s[None] - text).clamp(min=0)
    three = torch.stack([p // (w * w), p // w % w, p % w], dim=-1)
    three = torch.where((s[None] < text)[..., None], s[None, :, None], three + text[..., None])
    return three[..., :axes].contiguous().int()


def _tensors(case, heads, S, normal, gaps):
    """Tensors (B, S, H, D) for each of `heads`: slices of one packed projection where gaps, else each for itself."""
    B, D = case["B"], _head(case)
    if not gaps:
        return [normal(B, S, H, D) for H in heads]
    x = normal(B, S, sum(heads) * D)
    out, at = [], 0
    for H in heads:
        out.append(x[:, :, at:at + H * D].unflatten(-1, (H, D)))
        at += H * D
    return out


def _block_scale(a):
    """The smallest power of two s with a <= 448 s (at least 2^MIN_EXP), as FP32."""
    m, e = torch.frexp(a)                               # a = m 2^e, 1/2 <= m < 1
    e = torch.where(m > 0.875, e - 8, e - 9)            # 448 = 0.875 * 2^9
    e = torch.where(a > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return ((e.int() + 127) << 23).view(torch.float32)               # (a power, computed, may be off by a bit)


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _dtype(case)
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device=dev).normal_(generator=g)

    s = dict(case=case)
    if case["op"] == "rope":
        s["positions"] = _positions(case, dev, g)
        s["table"] = _angles(max(8192, case["S"] + 1), _sections(case), case["own_freqs"], dev)
        s["q"], s["k"] = _tensors(case, [case["Hq"], case["Hkv"]], case["S"], normal, case["packed"])
        return s
    if case["op"] == "store":
        n = 3 if case["packed"] else 1
        s["x"] = _tensors(case, [case["H"]] * n, case["S"], normal, case["packed"])[-1]
        s["x"].mul_(torch.empty((*s["x"].shape[:3], 1), device=dev).uniform_(0.1, 4.0, generator=g).to(dt))
        return s
    B, Hq, Hkv, Sq, Sk, D = (case[n] for n in ("B", "Hq", "Hkv", "Sq", "Sk", "D"))
    if case.get("packed"):
        q, k, v = _tensors(case, [Hq, Hkv, Hkv], Sq, normal, True)
    else:
        q, k, v = normal(B, Sq, Hq, D), normal(B, Sk, Hkv, D), normal(B, Sk, Hkv, D)
    s["do"] = normal(B, Sq, Hq, D).mul_(0.05)
    if case["op"] == "from8":
        for n, x in (("q", q), ("k", k), ("v", v)):
            scale = _block_scale(x.abs().amax(-1).float())
            s[n + "8"], s[n + "_scale"] = (x.float() / scale[..., None]).to(torch.float8_e4m3fn), scale
        return s
    s.update(q=q, k=k, v=v, mask=None)
    if case["masked"]:
        s["mask"] = torch.zeros((B, Sq, Sk), device=dev)
        s["mask"].masked_fill_(torch.rand((B, Sq, Sk), device=dev, generator=g) < 0.3, float("-inf"))
        s["mask"].masked_fill_((torch.arange(Sq, device=dev) % 97 == 96)[:, None], float("-inf"))
    s["o"], s["lse"] = _forward(case, q, k, v, s["mask"])            # what the forward pass has left
    return s


# ------------------------------------------------------------- plain forms

def _hidden(case, dev):
    """(Sq, Sk) truth values: key j is hidden from query i; None where nothing is."""
    if not case["causal"]:
        return None
    Sq, Sk = case["Sq"], case["Sk"]
    p = torch.arange(Sq, device=dev)[:, None] + (Sk - Sq)
    j = torch.arange(Sk, device=dev)
    h = j > p
    if case["window"]:
        h |= (j <= p - case["window"]) & (j >= case["sinks"])
    return h


def _logits(q, k, hide, mask):
    """Scaled and masked logits (G, Sq, Sk) of one K/V head in FP32."""
    x = torch.matmul(q * (1.0 / math.sqrt(q.shape[-1])), k.transpose(-1, -2))
    if mask is not None:
        x.add_(mask)
    if hide is not None:
        x.masked_fill_(hide, float("-inf"))
    return x


def _forward(case, q, k, v, mask):
    """o (B, Sq, Hq, D) of q's type and lse (B, Hq, Sq), one K/V head at a time. Rows without a key give 0 and -inf."""
    B, Sq, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    hide = _hidden(case, q.device)
    o = torch.empty((B, Sq, Hq, D), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, Hq, Sq), device=q.device)
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            x = _logits(q[b, :, heads].transpose(0, 1).float(), k[b, :, h].float(), hide,
                        None if mask is None else mask[b])
            m = x.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
            x.sub_(m).exp_()
            total = x.sum(-1, keepdim=True)
            y = torch.matmul(x, v[b, :, h].float()) / torch.where(total > 0, total, torch.ones_like(total))
            o[b, :, heads] = y.transpose(0, 1).to(q.dtype)
            lse[b, heads] = (m + total.log()).squeeze(-1)
    return o, lse


def _plain_backward(case, do, q, k, v, o, lse, mask):
    B, Sq, Hq, D = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    hide = _hidden(case, q.device)
    dq = torch.empty((B, Sq, Hq, D), dtype=q.dtype, device=q.device)
    dk, dv = (torch.empty((B, Sk, Hkv, D), dtype=q.dtype, device=q.device) for _ in range(2))
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            qf, of, gf = (t[b, :, heads].transpose(0, 1).float() for t in (q, o, do))
            kf, vf = k[b, :, h].float(), v[b, :, h].float()
            p = _logits(qf, kf, hide, None if mask is None else mask[b])
            l = lse[b, heads].masked_fill(lse[b, heads] == float("-inf"), float("inf"))
            p.sub_(l[..., None]).exp_()
            dv[b, :, h] = torch.matmul(p.transpose(-1, -2), gf).sum(0).to(q.dtype)
            ds = torch.matmul(gf, vf.transpose(-1, -2)).sub_((of * gf).sum(-1, keepdim=True)).mul_(p)
            dq[b, :, heads] = (torch.matmul(ds, kf) * scale).transpose(0, 1).to(q.dtype)
            dk[b, :, h] = (torch.matmul(ds.transpose(-1, -2), qf).sum(0) * scale).to(q.dtype)
    return dq, dk, dv


def _plain_rope(s):
    case, pos = s["case"], s["positions"].long()
    sections = _sections(case)
    axis = torch.repeat_interleave(torch.arange(len(sections), device=pos.device),
                                   torch.tensor(sections, device=pos.device))
    a = s["table"][pos[..., axis], torch.arange(sum(sections), device=pos.device)][:, :, None]    # (B, S, 1, D/2, 2)
    c, n = a[..., 0], -a[..., 1] if case["inverse"] else a[..., 1]

    def turn(x):
        x0, x1 = x[..., 0::2].float(), x[..., 1::2].float()
        return torch.stack([x0 * c - x1 * n, x1 * c + x0 * n], dim=-1).flatten(-2).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "rope":
            return _plain_rope(s)
        if case["op"] == "store":
            scale = _block_scale(s["x"].abs().amax(-1).float())
            return (s["x"].float() / scale[..., None]).to(torch.float8_e4m3fn), scale
        if case["op"] == "from8":
            q, k, v = ((s[n + "8"].float() * s[n + "_scale"][..., None]).to(_dtype(case)) for n in "qkv")
            o, lse = _forward(case, q, k, v, None)
            return _plain_backward(case, s["do"], q, k, v, o, lse, None)
        return _plain_backward(case, s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["mask"])
    import transformer_attention_02_gb300 as ta
    if case["op"] == "rope":
        return ta.rope_axes(s["q"], s["k"], s["table"], s["positions"], _sections(case), inverse=case["inverse"])
    if case["op"] == "store":
        return ta.checkpoint_store(s["x"])
    if case["op"] == "from8":
        return ta.attention_backward_checkpoint(
            s["do"], (s["q8"], s["q_scale"]), (s["k8"], s["k_scale"]), (s["v8"], s["v_scale"]), causal=case["causal"],
            window=case["window"], sinks=case["sinks"])
    return ta.attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], causal=case["causal"],
                                 mask=s["mask"], window=case["window"], sinks=case["sinks"])


# ------------------------------------------------------ the values in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "store":
        x = s["x"].double()
        top = x.abs().amax(-1)
        # from a power of two that is too small upwards, since a logarithm may miss where 448 s equals the maximum
        e = torch.log2(top.clamp(min=2.0 ** -120) / E4M3_MAX).floor() - 1
        scale = ((e.clamp(min=MIN_EXP).long() + 1023) << 52).view(torch.float64)
        for _ in range(3):
            scale = torch.where(scale * E4M3_MAX < top, 2 * scale, scale)
        return (x / scale[..., None]).to(torch.float8_e4m3fn), scale
    if case["op"] == "from8":
        q, k, v = (s[n + "8"].double() * s[n + "_scale"].double()[..., None] for n in "qkv")
        return _exact_backward(case, s["do"], q, k, v, None)
    return _exact_backward(case, s["do"], s["q"], s["k"], s["v"], s["mask"])


def _exact_rope(case, s):
    first, out = 0, [torch.empty(t.shape, dtype=torch.float64, device=t.device) for t in (s["q"], s["k"])]
    for a, n in enumerate(_sections(case)):
        turn = torch.view_as_complex(s["table"].double()[:, first:first + n].contiguous())[s["positions"][..., a].long()]
        if case["inverse"]:
            turn = turn.conj()
        part = slice(2 * first, 2 * (first + n))
        for x, y in zip((s["q"], s["k"]), out):
            z = torch.view_as_complex(x[..., part].double().unflatten(-1, (n, 2)).contiguous())
            y[..., part] = torch.view_as_real(z * turn[:, :, None]).flatten(-2)
        first += n
    return tuple(out)


def _exact_backward(case, do, q, k, v, mask):
    """From the definition, 1024 queries of one head at a time, over the keys that they see."""
    if case["B"] * case["Hq"] * case["D"] * _visible(case)[0] > 2 ** 39:
        return None
    B, Sq, Hq, D = q.shape
    Sk, G, dev = k.shape[1], Hq // k.shape[2], q.device
    dq = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    dk, dv = (torch.zeros(k.shape, dtype=torch.float64, device=dev) for _ in range(2))
    all_keys = torch.arange(Sk, device=dev)
    for i0 in range(0, Sq, 1024):
        i1 = min(Sq, i0 + 1024)
        keys = all_keys
        see = torch.ones((i1 - i0, Sk), dtype=torch.bool, device=dev)
        if case["causal"]:
            dist = torch.arange(i0, i1, device=dev)[:, None] + (Sk - Sq) - all_keys
            see = dist >= 0
            if case["window"]:
                see &= (dist < case["window"]) | (all_keys < case["sinks"])
            keys = all_keys[see.any(0)]
            see = see[:, keys]
        if len(keys) == 0:
            continue
        whole = len(keys) == Sk
        for b in range(B):
            for h in range(Hq):
                pick = (lambda t: t[b, :, h // G]) if whole else (lambda t: t[b, keys, h // G])
                qq, g = q[b, i0:i1, h].double() / math.sqrt(D), do[b, i0:i1, h].double()
                kk, vv = pick(k).double(), pick(v).double()
                z = qq @ kk.T
                if mask is not None:
                    z += mask[b, i0:i1, keys].double()
                z.masked_fill_(~see, float("-inf"))
                p = torch.nan_to_num(torch.softmax(z, dim=-1), nan=0.0)      # a row without keys has no probabilities
                dp = g @ vv.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True))
                dq[b, i0:i1, h] = ds @ kk / math.sqrt(D)
                dk[b, :, h // G].index_add_(0, keys, ds.T @ qq)
                dv[b, :, h // G].index_add_(0, keys, p.T @ g)
    return dq, dk, dv
