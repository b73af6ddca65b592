"""The attention's backward pass in 64 bits, by the formulas, and how far the kernels may be from it.

The bounds are worst cases, element by element, from what the kernels round: P and dS to the tensors' type (half a step
each, eps / 2 relative; for fp16 2^-25 at least), the gradients on their way out, the forward pass's output, which enters
delta, and FP32 sums and exponentials (2^-24 a step; the exponent's own error grows with the logit).
"""
import math

import torch

LOG2E = float(torch.tensor(1.4426950408889634))


def visible(Sq, Sk, causal, window=0, sinks=0, device="cpu"):
    see = torch.ones((Sq, Sk), dtype=torch.bool, device=device)
    if causal:
        p = torch.arange(Sq, device=device)[:, None] + (Sk - Sq)
        j = torch.arange(Sk, device=device)
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
    return see


def _probs(q, k, scale, see, mask, fp32_logits=True):
    z = torch.einsum("bihd,bjhd->bhij", q, k) * scale
    if mask is not None and not fp32_logits:
        z = z + mask.double()[:, None]
    elif mask is not None:
        # Masked logits are FP32 numbers in log2 units, as in the forward pass: of logits that a mask moves by 1e9, only
        # multiples of 128 are left. This rounding is part of the operator, so the reference makes it too.
        z = ((mask.double()[:, None] * LOG2E + (z.float() * LOG2E).double()).float().double() / LOG2E)
    z = z.masked_fill(~see, float("-inf"))
    m = z.amax(-1, keepdim=True) if z.shape[-1] else z.new_full((*z.shape[:-1], 1), float("-inf"))
    e = (z - m.masked_fill(m == float("-inf"), 0)).exp()
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    return z, p, (m + total.log()).squeeze(-1)


def forward(q, k, v, *, causal=False, mask=None, window=0, sinks=0, scale=None):
    """o (B, Sq, Hq, D) and lse (B, Hq, Sq) in FP64."""
    Sq, D, G, Sk = q.shape[1], q.shape[3], q.shape[2] // k.shape[2], k.shape[1]
    kk, vv = (t.double().repeat_interleave(G, dim=2) for t in (k, v))
    _, p, lse = _probs(q.double(), kk, scale or 1 / math.sqrt(D), visible(Sq, Sk, causal, window, sinks, q.device), mask,
                       q.dtype != torch.float64)
    return torch.einsum("bhij,bjhd->bihd", p, vv).contiguous(), lse


def backward(d_o, q, k, v, *, causal=False, mask=None, window=0, sinks=0, scale=None):
    """((dq, dk, dv), (their bounds)) in FP64, for inputs of the type of q."""
    dtype = q.dtype
    B, Sq, Hq, D = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    scale = scale or 1 / math.sqrt(D)
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0            # half a step of the subnormal range
    flush = 2.0 ** -126                                             # FP32 exponentials below it become zero
    u = 2.0 ** -24
    g, qq = d_o.double(), q.double()
    kk, vv = (t.double().repeat_interleave(G, dim=2) for t in (k, v))
    z, p, _ = _probs(qq, kk, scale, visible(Sq, Sk, causal, window, sinks, q.device), mask, dtype != torch.float64)
    o = torch.einsum("bhij,bjhd->bihd", p, vv)
    dp = torch.einsum("bihd,bjhd->bhij", g, vv)
    delta = torch.einsum("bihd,bihd->bhi", g, o)
    ds = p * (dp - delta[..., None])

    def heads(x):                                                    # the sum over the query heads of a K/V head
        return x.unflatten(2, (Hkv, G)).sum(3)

    dq = torch.einsum("bhij,bjhd->bihd", ds, kk) * scale
    dk = heads(torch.einsum("bhij,bihd->bjhd", ds, qq)) * scale
    dv = heads(torch.einsum("bhij,bihd->bjhd", p, g))

    # FP32: a logit is off by its products' sum, the scaled sum, the mask's and the statistics' rounding (lse and the
    # logits are as large as `big`); P by the exponential of that and of ex2's own 2 steps.
    big = torch.where(z.isinf(), torch.zeros_like(z), z.abs())
    spread = torch.einsum("bihd,bjhd->bhij", qq.abs(), kk.abs()) * scale
    if mask is not None:                                             # statistics are found in the same arithmetic, so
        big = torch.einsum("bihd,bjhd->bhij", qq.abs(), kk.abs()) * scale + 8   # a row's shift cancels
        # The rounding above may fall the other way where a sum lies next to a border: by u |z| where that is less than the
        # sums' own spacing; past 2^20 all of a row's logits are a few numbers, and both sides find the same ones.
        big = big + torch.where(z.abs() < 2 ** 20, z.abs(), torch.zeros_like(z))
    rel = 4 * u + 8 * u * spread + 6 * u * (big + big.amax(-1, keepdim=True) if Sk else big)
    ddelta = (half + 8 * u) * torch.einsum("bihd,bihd->bhi", g.abs(), o.abs())[..., None]
    ddp = 8 * u * torch.einsum("bihd,bjhd->bhij", g.abs(), vv.abs())
    e_p = p * (half + rel) + tiny * (p > 0) + flush
    e_ds = ds.abs() * (half + 2 * rel) + p * (ddelta + ddp) + tiny * (p > 0) + flush * (1 + (dp - delta[..., None]).abs())
    out = half + 16 * u

    def bound(err, x, y):
        return err * 1.01 + out * x.abs() + tiny + flush

    b_dq = bound(torch.einsum("bhij,bjhd->bihd", e_ds + 4 * u * ds.abs(), kk.abs()) * scale, dq, dtype)
    b_dk = bound(heads(torch.einsum("bhij,bihd->bjhd", e_ds + 4 * u * ds.abs(), qq.abs())) * scale, dk, dtype)
    b_dv = bound(heads(torch.einsum("bhij,bihd->bjhd", e_p + 4 * u * p, g.abs())), dv, dtype)
    return (dq, dk, dv), (b_dq, b_dk, b_dv)


def check(got, want, bounds, label=""):
    for name, a, w, b in zip(("dq", "dk", "dv") if len(got) == 3 else ("gradient",), got, want, bounds):
        assert bool(torch.isfinite(a).all()), f"{label} {name}: not finite"
        err = (a.double() - w).abs()
        worst = float((err / b.clamp(min=1e-300)).max()) if err.numel() else 0.0
        assert bool((err <= b).all()), f"{label} {name}: {worst:.2f} of the bound, {float(err.max()):.3e}"
