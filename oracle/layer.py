"""Plain 64-bit forms of the operators around the attention (numpy, loops over
sequences): the paged cache, its attention, and the layer norm with its gate
and residual.  Test infrastructure; shares no code with the library.
"""
from __future__ import annotations

import numpy as np


def f64(t) -> np.ndarray:
    """A torch tensor (any float type) or array as float64."""
    if hasattr(t, "detach"):
        t = t.detach().cpu().double().numpy()
    return np.asarray(t, dtype=np.float64)


def rotate(x: np.ndarray, pos: int, table: np.ndarray, pairs: bool) -> np.ndarray:
    """Rotate the first table.shape[1] channels of x (heads, d) to position pos."""
    y = x.copy()
    half = table.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, half + i)
        c, s = table[pos, i], table[pos, half + i]
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def append(k_pages, v_pages, k, v, q, q_offsets, kv_lens, page_table, num_targets=None, table=None,
           pairs=False):
    """(k_pages, v_pages, q_out) in float64 after the append; rows that no
    sequence holds are NaN in q_out."""
    kp, vp = f64(k_pages), f64(v_pages)
    k, v, q = f64(k), f64(v), f64(q)
    q_out = np.full_like(q, np.nan)
    ps = kp.shape[1]
    for b in range(len(kv_lens)):
        n = int(q_offsets[b + 1] - q_offsets[b])
        hist = int(kv_lens[b]) - (0 if num_targets is None else int(num_targets[b]))
        for i in range(n):
            t, p = int(q_offsets[b]) + i, int(kv_lens[b]) - n + i
            page, slot = int(page_table[b, p // ps]), p % ps
            kk, qq = k[t], q[t]
            if table is not None:
                kk, qq = (rotate(x, min(p, hist), f64(table), pairs) for x in (kk, qq))
            kp[page, slot], vp[page, slot], q_out[t] = kk, v[t], qq
    return kp, vp, q_out


def attention(k_pages, v_pages, q, q_offsets, kv_lens, page_table, alpha, inv_n, num_targets=None):
    """(out, bound): the attention over the cache, and for each output the sum
    that its rounding errors scale with (NaN where no sequence holds the row).

    bound = inv_n * sum_j e_j |v_j| over the kept keys, e_j the error of one
    p_j = silu(x_j): tanh.approx.f32 (2^-16 relative, as measured) on
    h = x / 2, the split of p into two bf16 (2^-17 p), the fp32 dot product
    (d + 8 roundings of 2^-24 on sum_c |q_c k_c|, slope of silu <= 1.1) and
    the fp32 sums over keys (one rounding a 16-key product and 64 joins).
    """
    q = f64(q)
    out = np.full(q.shape, np.nan)
    bound = np.full(q.shape, np.nan)
    ps, d = k_pages.shape[1], q.shape[2]
    for b in range(len(kv_lens)):
        n, kv = int(q_offsets[b + 1] - q_offsets[b]), int(kv_lens[b])
        if n == 0:
            continue
        pages = np.asarray(page_table[b, :(kv + ps - 1) // ps], dtype=np.int64)
        k = f64(k_pages[pages]).reshape(-1, q.shape[1], d)[:kv]
        v = f64(v_pages[pages]).reshape(-1, q.shape[1], d)[:kv]
        hist = kv - (0 if num_targets is None else int(num_targets[b]))
        for i in range(n):
            t, p = int(q_offsets[b]) + i, kv - n + i
            kept = [j for j in range(p + 1) if j < hist or j == p]
            for h in range(q.shape[1]):
                kk, vv = k[kept, h], v[kept, h]
                x = alpha * (kk @ q[t, h])
                with np.errstate(over="ignore"):
                    w = x / (1.0 + np.exp(-x))
                out[t, h] = inv_n * (w @ vv)
                dot = abs(alpha) * (np.abs(kk) @ np.abs(q[t, h]))
                e = 2.0 ** -16 * np.abs(x) + 2.0 ** -17 * np.abs(w) + 1.1 * (d + 8) * 2.0 ** -24 * dot \
                    + (len(kept) / 16 + 64) * 2.0 ** -24 * np.abs(w)
                bound[t, h] = abs(inv_n) * (e @ np.abs(vv))
    return out, bound


def norm_fwd(x, gamma, beta, eps, u=None, residual=None, scale=1.0):
    """(y, z) in float64."""
    z = f64(x) * scale + f64(residual) if residual is not None else f64(x)
    xhat, _ = standard(z, eps)
    y = xhat * f64(gamma) + f64(beta)
    return (y if u is None else y * f64(u)), z


def standard(z, eps):
    dev = z - z.mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt((dev ** 2).mean(axis=1, keepdims=True) + eps)
    return dev * rstd, rstd


def norm_bwd(dy, z, gamma, beta, eps, u=None, dz_in=None, scale=1.0):
    """dict of dz, dx, du, dgamma, dbeta in float64."""
    z, dy, gamma, beta = f64(z), f64(dy), f64(gamma), f64(beta)
    xhat, rstd = standard(z, eps)
    g = dy if u is None else dy * f64(u)
    a = g * gamma
    dz = rstd * (a - a.mean(axis=1, keepdims=True) - xhat * (a * xhat).mean(axis=1, keepdims=True))
    if dz_in is not None:
        dz = dz + f64(dz_in)
    return dict(dz=dz, dx=scale * dz, du=dy * (xhat * gamma + beta), dgamma=(g * xhat).sum(axis=0),
                dbeta=g.sum(axis=0))


# ------------------------------------------------------ a cache of 4-bit codes
SCALES = np.array([(8 + j % 8) * 2.0 ** (j // 8 - 23) for j in range(256)])


def q4_codes(x):
    """(codes, scale numbers) of x (..., d): the integer nearest to x / s, ties
    away from zero, s the first scale with 7 s >= the group's largest |x|."""
    g = f64(x)
    g = np.where(np.isnan(g), 0.0, np.where(np.isinf(g), np.sign(g) * (2.0 - 2.0 ** -7) * 2.0 ** 127, g))
    g = g.reshape(*g.shape[:-1], -1, 16)
    most = np.abs(g).max(axis=-1)
    j = np.minimum(np.searchsorted(7 * SCALES, most), 255)  # the first that holds it
    q = np.abs(g) / SCALES[j][..., None]
    code = (np.sign(g) * np.minimum(np.floor(q + 0.5), 7)).astype(np.int64)
    return code.reshape(*code.shape[:-2], -1), j


def q4_values(code, j):
    return (code.reshape(*j.shape, 16) * SCALES[j][..., None]).reshape(code.shape)


def q4_held(x):
    """What the cache holds for x (..., d)."""
    return q4_values(*q4_codes(x))


def _q4_places(page, heads, d):
    """Byte places in a page: (keys' codes, values' codes), each (page, heads, d),
    with the bit that a channel's nibble starts at, and the scales' (page,
    heads, d / 16)."""
    t = min(page, 128)
    p, h, c = (np.arange(n) for n in (page, heads, d))
    tile = (h[None, :] * (page // t) + p[:, None] // t) * (t * d * 9 // 8)
    bit = 32 * (c // 8) + 16 * (c % 2) + 4 * (c % 8 // 2)
    row = (p % t)[:, None, None]
    codes = [tile[..., None] + w * t * d // 2 + row * (d // 2) + bit // 8 for w in (0, 1)]
    g = np.arange(d // 16)
    scales = [tile[..., None] + t * d + w * t * d // 16 + row * (d // 16) + g for w in (0, 1)]
    return codes, bit % 8, scales


def q4_pack(k_pages, v_pages):
    """Pages of bytes (num_pages, bytes) that hold the values (num_pages, page, heads, d)."""
    n, page, heads, d = k_pages.shape
    codes, shift, scales = _q4_places(page, heads, d)
    out = np.zeros((n, page * heads * d * 9 // 8), dtype=np.uint8)
    for x, at, sat in zip((k_pages, v_pages), codes, scales):
        code, j = q4_codes(x)
        for s in (0, 4):  # no byte twice in one assignment
            out[:, at[..., shift == s]] |= ((code[..., shift == s] & 15) << s).astype(np.uint8)
        out[:, sat] = j
    return out


def q4_unpack(pages, page, heads, d):
    """(keys, values) in float64 (num_pages, page, heads, d) of pages of bytes."""
    pages = np.asarray(pages)
    codes, shift, scales = _q4_places(page, heads, d)
    out = []
    for at, sat in zip(codes, scales):
        code = pages[:, at].astype(np.int64) >> shift & 15
        out.append(q4_values(np.where(code > 7, code - 16, code), pages[:, sat].astype(np.int64)))
    return out
