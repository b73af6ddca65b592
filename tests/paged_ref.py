"""Plain 64-bit reference of the paged cache's operators for the tests: one sequence and one head at a time, in
NumPy, from the definitions in include/attn.h. Shares no code with the library."""
import numpy as np
import torch

E4M3_MAX = 448.0


def step(t):
    """Half a rounding step of a type, relative to the value."""
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rotate(x, pos, base=10000.0):
    """x (n, H, D) in FP64 with row r at pos[r]; interleaved pairs."""
    D = x.shape[-1]
    ang = np.asarray(pos, np.float64)[:, None] * base ** (-2.0 * np.arange(D // 2) / D)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y = np.empty_like(x)
    y[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    y[..., 1::2] = x[..., 1::2] * c + x[..., 0::2] * s
    return y


def block_scale(a):
    """Smallest power of two s >= 2^-100 with a <= 448 s."""
    e = -100
    while a > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def tokens(cache, scale, table_row, n, page):
    """The first n tokens' values (n, Hkv, D) in FP64 of a sequence's pages."""
    ids = table_row[:-(-n // page)].astype(np.int64)
    x = f64(cache[torch.as_tensor(ids, device=cache.device)] if cache.element_size() > 1 else
            cache.view(torch.uint8)[torch.as_tensor(ids, device=cache.device)].view(cache.dtype))
    if scale is not None:
        x = x * f64(scale)[ids][:, :, None, None]
    return x.transpose(0, 2, 1, 3).reshape(-1, cache.shape[1], cache.shape[3])[:n]


def attend(q, k, v, pos, scale, window, sinks):
    """q (n, Hq, D) at pos (n), k and v (L, Hkv, D): o (n, Hq, D), lse (Hq, n), and for the bounds the weighted |v|
    (n, Hq, D) and each row's largest sum of |q_d k_d| times the scale (n, Hq). Hidden keys' values never enter."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    j = np.arange(L)
    o, lse = np.zeros(q.shape), np.full((Hq, n), -np.inf)
    a, mag = np.zeros(q.shape), np.zeros((n, Hq))
    for i in range(n):
        see = j <= pos[i]
        if window:
            see &= (j > pos[i] - window) | (j < sinks)
        if not see.any():
            continue
        for h in range(Hq):
            kk, vv = k[see, h // (Hq // Hkv)], v[see, h // (Hq // Hkv)]
            z = scale * (kk @ q[i, h])
            m = z.max()
            w = np.exp(z - m)
            lse[h, i] = m + np.log(w.sum())
            w /= w.sum()
            o[i, h], a[i, h] = w @ vv, w @ np.abs(vv)
            mag[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return o, lse, a, mag


def check_rows(o, lse, want, out_step, p_step, D, n_keys, v_top, label=""):
    """o (n, Hq, D) and lse (Hq, n) against attend()'s result.

    |o - o*| <= out_step |o*|                      the output's one rounding
              + (p_step + 2 dz + 2^-18) sum p|v|   the weights' rounding to 16 bits, an error dz in a logit (it moves a
                                                   weight and the normaliser), the approximate exponential and FP32 sums
              + n 2^-24 v_top                      weights below the 16-bit normal range (half a subnormal step, 2^-25,
                                                   twice for the sum's side)
    dz = (D + 8) 2^-24 * max sum |q_d k_d| scale: D products summed in FP32, then three FP32 roundings of the logit.
    """
    wo, wl, a, mag = want
    dz = (D + 8) * 2.0 ** -24 * mag
    tol = out_step * np.abs(wo) + (p_step + 2 * dz + 2.0 ** -18)[..., None] * a + n_keys * 2.0 ** -24 * v_top + 1e-30
    assert np.isfinite(o).all(), f"{label}: non-finite O"
    bad = np.abs(o - wo) / tol
    assert bad.max(initial=0.0) <= 1.0, f"{label}: O off by {bad.max():.2f} of its bound"
    empty = ~np.isfinite(wl)
    assert np.all(lse[empty] == -np.inf) and np.all(o[empty.T] == 0.0), f"{label}: rows without a key"
    lt = dz.T + 2.0 ** -18 + 2.0 ** -21 * np.abs(np.where(empty, 0, wl))
    le = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, wl)) / lt
    assert le.max(initial=0.0) <= 1.0, f"{label}: LSE off by {le.max():.2f} of its bound"
