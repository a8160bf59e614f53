"""Oracle of the attention side: head norms with rotation, the 4-bit cache's
codes and layout, attention over the cache and over packed prompts (numpy,
float64)."""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def norm_rope(x, w, eps, positions, table, R, interleaved):
    """(y, size): y of heads x [T, NH, D] in float64, and per element the sum
    of the magnitudes that its last addition joins (the scale of its float32
    error).  w None: no norm."""
    z = np.asarray(x, np.float64)
    if w is not None:
        z = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y, size = z.copy(), np.abs(z)
    half = R // 2
    for t, p in enumerate(np.clip(positions, 0, table.shape[0] - 1)):
        for i in range(half):
            c, s = float(table[p, i]), float(table[p, half + i])
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            za, zb = z[t, :, a], z[t, :, b]
            y[t, :, a], size[t, :, a] = za * c - zb * s, np.abs(za * c) + np.abs(zb * s)
            y[t, :, b], size[t, :, b] = zb * c + za * s, np.abs(zb * c) + np.abs(za * s)
    return y, size


def quantise(x):
    """(codes 0..15, scale bytes) of [..., D] finite or not: groups of 32."""
    g = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], -1, 32)
    amax = np.abs(g).max(-1)
    good = np.isfinite(amax)
    e = np.full(amax.shape, -125)
    for k in range(-125, 125):                     # the smallest that holds amax
        e = np.where(amax > 7.0 * 2.0 ** k, k + 1, e)
    a = np.where(good[..., None], np.abs(g), 0.0) / 2.0 ** e[..., None]
    dist = np.abs(a[..., None] - E2M1)
    # the nearest; of two the even code
    code = np.where(dist[..., ::2].min(-1) <= dist[..., 1::2].min(-1),
                    2 * dist[..., ::2].argmin(-1), 2 * dist[..., 1::2].argmin(-1) + 1)
    code = code + 8 * np.signbit(g)
    return code.reshape(np.shape(x)), np.where(good, e + 127, 255)


def values(codes, scales):
    """What codes [..., D] with scale bytes [..., D / 32] stand for."""
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (np.asarray(scales, np.float64) - 127))
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(codes.shape)


def k_place(D, token, d):
    """(byte, shift) of the code of feature d of a tile's token, K part."""
    return token * (D // 2) + d // 2, 4 * (d % 2)


def v_place(D, token, d):
    chunk, r = d // 128, d % 128
    w = 8 if (chunk + 1) * 128 <= D else 4          # features side by side
    return (8 * D + D // 2 + chunk * 1024 + (((token // 4) * 16 + r // w) * 4 + token % 4) * (w // 2)
            + r % w // 2, 4 * (d % 2))


def k_scale_place(D, token, g):
    return 8 * D + token * (D // 32) + g


def v_scale_place(D, token, g):
    return 16 * D + D // 2 + ((token // 4) * (D // 32) + g) * 4 + token % 4


def put(pages, page, h, slot, k, v):
    """Writes one token's key and value [D] into pages [P, NKV, tiles, 17 D]."""
    D = len(k)
    tile, t = pages[page, h, slot // 16], slot % 16
    for x, place, scale_place in ((k, k_place, k_scale_place), (v, v_place, v_scale_place)):
        codes, scales = quantise(x)
        for d in range(D):
            byte, shift = place(D, t, d)
            tile[byte] = (int(tile[byte]) & ~(15 << shift)) | int(codes[d]) << shift
        for g in range(D // 32):
            tile[scale_place(D, t, g)] = scales[g]


def get(pages, page, h, slot):
    """One token's (key, value) [D] as float64."""
    tile, t = pages[page, h, slot // 16], slot % 16
    D = len(tile) // 17
    out = []
    for place, scale_place in ((k_place, k_scale_place), (v_place, v_scale_place)):
        codes = np.array([int(tile[place(D, t, d)[0]]) >> place(D, t, d)[1] & 15 for d in range(D)])
        scales = np.array([tile[scale_place(D, t, g)] for g in range(D // 32)])
        out.append(values(codes, scales))
    return out


def attend(q, k, v, scale, sees=None):
    """(out, lse, spread, reach) of queries [n, D] over keys and values
    [m, D]: spread = sum p |v| and reach = the largest sum |q||k| * scale are
    the sizes that errors are measured against.  sees [n]: how many keys each
    query sees (default: all)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, m = len(q), len(k)
    sees = np.full(n, m) if sees is None else np.clip(sees, 0, m)
    out = np.zeros((n, v.shape[1]))
    spread, lse, reach = np.zeros_like(out), np.full(n, -np.inf), np.zeros(n)
    for i in range(n):
        c = int(sees[i])
        if c == 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            s = k[:c] @ q[i] * scale
            top = s.max()
            p = np.exp(s - top)
            z = p.sum()
            p /= z
            out[i], spread[i] = p @ v[:c], p @ np.abs(v[:c])
            lse[i] = top + np.log(z)
            reach[i] = (np.abs(k[:c]) @ np.abs(q[i])).max() * scale
    return out, lse, spread, reach
