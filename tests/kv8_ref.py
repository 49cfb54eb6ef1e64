"""64-bit restatement of the 8-bit paged cache (attn_kv8_write, attn_kv8_read) and of rotary
positions (attn_rope) in numpy, group by group and pair by pair, for the tests.

Codes are uint8 arrays [pages, P, H, D], scales float32 [pages, H, P / G]."""
import math

import numpy as np

FLOOR = 2.0 ** -100
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)])


def values(codes, fmt):
    """float64 values of uint8 codes (before the scale)."""
    if fmt == "int8":
        return codes.view(np.int8).astype(np.float64)
    return np.where(codes & 0x80, -1.0, 1.0) * E4M3[codes & 0x7f]


def encode(x, fmt):
    """uint8 codes nearest to float64 x, ties to the even code."""
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x), 448.0)
    table = E4M3[:127]
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - a, a - table[lo]
    i = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (i | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def new_scale(amax, fmt):
    if not math.isfinite(amax):
        return np.float32(np.nan)
    if fmt == "int8":
        return np.float32(max(float(np.float32(amax / 127.0)), FLOOR))
    return np.float32(max(2.0 ** math.ceil(math.log2(amax / 448.0)) if amax > 0 else 0.0, FLOOR))


def write_one(x, codes, scales, table, lens, offs, fmt, G):
    """Writes float64 x [tokens, H, D] into codes and scales, in place."""
    P, H = codes.shape[1:3]
    T, pages, max_pages = x.shape[0], codes.shape[0], table.shape[1]
    for s in range(len(lens)):
        lo = min(max(int(offs[s]), 0), T)
        n = min(max(int(offs[s + 1]), lo), T) - lo
        L = min(max(int(lens[s]), 0), max_pages * P)
        first = max(L - n, 0)
        g = first // G
        while n and g * G < L:
            a, b = max(first, g * G), min(L, (g + 1) * G)
            page, held = int(table[s, g * G // P]), a - g * G
            if 0 <= page < pages:
                r, part = g * G % P, x[lo + a - (L - n):lo + b - (L - n)]
                for h in range(H):
                    S = new_scale(float(np.max(np.abs(part[:, h]))) if np.isfinite(part[:, h]).all() else np.inf, fmt)
                    if held:
                        old = scales[page, h, r // G]
                        S = np.float32(np.nan) if np.isnan(old) or np.isnan(S) else max(old, S)
                        if S > old:
                            c = codes[page, r:r + held, h]
                            codes[page, r:r + held, h] = encode(values(c, fmt) * float(old) / float(S), fmt)
                    scales[page, h, r // G] = S
                    codes[page, r + held:r + b - g * G, h] = 0 if np.isnan(S) else encode(part[:, h] / float(S), fmt)
            g += 1


def read_all(codes, scales, fmt):
    """float64 values of a whole cache [pages, P, H, D]."""
    per = scales.shape[2]
    sc = np.repeat(scales.astype(np.float64), codes.shape[1] // per, axis=2)  # [pages, H, P]
    return values(codes, fmt) * sc.transpose(0, 2, 1)[..., None]


def read_rows(codes, scales, table, lens, offs, rows, fmt, starts=None, fill=np.nan):
    """float64 [rows, H, D]; ``fill`` in rows of no sequence."""
    v = read_all(codes, scales, fmt)
    pages, P, H, D = codes.shape
    out = np.full((rows, H, D), fill)
    for s in range(len(lens)):
        lo = min(max(int(offs[s]), 0), rows)
        hi = min(max(int(offs[s + 1]), lo), rows)
        L = min(max(int(lens[s]), 0), table.shape[1] * P)
        for i in range(hi - lo):
            j = i + (int(starts[s]) if starts is not None else 0)
            page = int(table[s, j // P]) if 0 <= j < L else -1
            out[lo + i] = v[page, j % P] if 0 <= page < pages else 0.0
    return out


def attention(q, k, v, table, lens, offs, positions=None, causal=True, scale=1.0):
    """float64 attention over float64 caches k, v [pages, P, H, D]: the output, the natural
    log-sum-exp, sum_j p_j |v_j| of each output, and the largest sum |q||k| scale of a row."""
    nq, Hq, D = q.shape
    pages, P, H, _ = k.shape
    out, lse = np.full((nq, Hq, D), np.nan), np.full((nq, Hq), -np.inf)
    mag, big = np.zeros((nq, Hq, D)), np.zeros((nq, Hq))
    for s in range(len(lens)):
        lo, hi = int(offs[s]), int(offs[s + 1])
        L = min(int(lens[s]), table.shape[1] * P)
        j = np.arange(L)
        page = table[s, j // P] if L else np.zeros(0, int)
        ok = (page >= 0) & (page < pages)
        kk = np.where(ok[:, None, None], k[np.where(ok, page, 0), j % P], 0.0)
        vv = np.where(ok[:, None, None], v[np.where(ok, page, 0), j % P], 0.0)
        for i in range(lo, hi):
            pos = int(positions[i]) if positions is not None else L - (hi - lo) + (i - lo)
            n = min(L, pos + 1) if causal else L
            if n <= 0:
                continue
            for h in range(Hq):
                hk = h // (Hq // H)
                t = kk[:n, hk] @ q[i, h] * scale
                m = t.max()
                p = np.exp(t - m)
                z = p.sum()
                out[i, h] = p @ vv[:n, hk] / z
                mag[i, h] = p @ np.abs(vv[:n, hk]) / z
                big[i, h] = (np.abs(kk[:n, hk]) @ np.abs(q[i, h])).max() * scale
                lse[i, h] = m + math.log(z)
    return out, lse, mag, big


def rope(x, pos, freq, layout, mscale=1.0, inverse=False):
    """float64 x [tokens, H, D] turned by positions [tokens]."""
    a = pos.astype(np.float64)[:, None] * freq[None, :] * (-1 if inverse else 1)
    c, s = np.cos(a)[:, None] * mscale, np.sin(a)[:, None] * mscale
    n, y = len(freq), x.copy()
    i, j = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y
