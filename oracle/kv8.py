"""Plain fp64 oracle of prompt attention and of the cache in 8 bits: e4m3
rounding, the factor of a page, appending rows, and attention over rows.
"""

import math

import numpy as np

PAGE = 16
TOP = 448.0


def _e4m3_values():
    """The value of each of the 256 codes, from the format's definition."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v[c] = (-1.0) ** s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        if e == 15 and m == 7:
            v[c] = math.nan
    return v


E4M3 = _e4m3_values()


def to_e4m3(x):
    """Codes of the nearest values (ties to the even code); what lies beyond 448,
    infinities among it, becomes 448 of its sign, NaN the code 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    pos = E4M3[:127]                                    # 0 .. 448, ascending
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=TOP, neginf=-TOP)), TOP)
    hi = np.minimum(np.searchsorted(pos, a), 126)       # first value >= a
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(pos[hi] == a, hi, code)
    code = code + np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def page_scale(rows):
    """The smallest power of two, at least 2^-126, with |x| <= 448 * it for every
    finite x of rows (bf16 values)."""
    rows = np.abs(np.asarray(rows, dtype=np.float64))
    rows = rows[np.isfinite(rows)]
    s = 2.0 ** -126
    while rows.size and rows.max() > TOP * s:
        s *= 2
    return s


def kv8_append(codes, scales, base, new):
    """One sequence's logical rows of one pool: codes uint8 [Hkv][capacity][d] and
    scales [Hkv][capacity / 16] (both changed), new [n][Hkv][d] bf16 values at
    positions base, base + 1, ..."""
    new = np.asarray(new, dtype=np.float64)
    done = 0
    while done < len(new):
        at = base + done
        page, r0 = at // PAGE, at % PAGE
        take = min(PAGE - r0, len(new) - done)
        for g in range(codes.shape[0]):
            rows = new[done: done + take, g]
            s, first = page_scale(rows), page * PAGE
            if r0:
                old = scales[g, page]
                s = max(s, old)
                codes[g, first: at] = to_e4m3(E4M3[codes[g, first: at]] * (old / s))
            codes[g, at: at + take] = to_e4m3(rows / s)
            scales[g, page] = s
        done += take


def kv8_rows(codes, scales):
    """Values [Hkv][capacity][d] of logical rows."""
    return E4M3[codes] * np.repeat(scales, PAGE, axis=1)[..., None]


def attend(q, K, V, scale):
    """One row q [d] over K, V [n][d]: (out [d], lse, the average of |V|)."""
    if len(K) == 0:
        return np.zeros(V.shape[1]), -math.inf, np.zeros(V.shape[1])
    z = scale * (K @ q)
    m = z.max()
    w = np.exp(z - m)
    return w / w.sum() @ V, m + math.log(w.sum()), w / w.sum() @ np.abs(V)


def prompt_attention(q, k, v, seq_start, scale):
    """q [N][H][d], k, v [N][Hkv][d] packed; (out, lse, mag), rows of no sequence NaN."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    N, H, d = q.shape
    G = H // k.shape[1]
    out, lse, mag = np.full((N, H, d), np.nan), np.full((N, H), np.nan), np.full((N, H, d), np.nan)
    for s0, s1 in zip(seq_start[:-1], seq_start[1:]):
        n = s1 - s0
        if n == 0:
            continue
        later = np.triu(np.ones((n, n), dtype=bool), 1)
        for h in range(H):
            K, V = k[s0:s1, h // G], v[s0:s1, h // G]
            z = np.where(later, -math.inf, scale * (q[s0:s1, h] @ K.T))
            m = z.max(1, keepdims=True)
            w = np.exp(z - m)
            total = w.sum(1, keepdims=True)
            out[s0:s1, h], mag[s0:s1, h] = (w / total) @ V, (w / total) @ np.abs(V)
            lse[s0:s1, h] = (m + np.log(total))[:, 0]
    return out, lse, mag
