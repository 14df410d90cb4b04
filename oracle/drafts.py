"""Plain fp64 oracle of the new-token, draft and branch operations around the
paged cache: per-head norm and rotation, attention of a draft tree, the
compaction of its accepted path, and pages shared between branches.
"""

import math

import numpy as np

PAGE = 16


def norm_rope(x, weight, eps, cos_sin, pos, sections=None, interleaved=False):
    """Per-head RMS norm (weight None: none) and rotation, from the formulas.

    x [B][T][h][d]; weight [d] or None; cos_sin [n_pos][rot / 2][2] or None;
    pos [B][T], or with sections (pairs per axis) [axes][B][T].  Pair p is
    elements (p, rot / 2 + p), or (2p, 2p + 1) when interleaved.
    """
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    if cos_sin is None:
        return y
    cos_sin = np.asarray(cos_sin, dtype=np.float64)
    pos = np.asarray(pos)
    half = cos_sin.shape[1]
    if sections is None:
        pos, sections = pos.reshape((1,) + pos.shape[-2:]), [half]
    axis = np.repeat(np.arange(len(sections)), sections)
    out = y.copy()
    for b in range(x.shape[0]):
        for t in range(x.shape[1]):
            for p in range(half):
                c, s = cos_sin[pos[axis[p], b, t], p]
                i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
                out[b, t, :, i] = y[b, t, :, i] * c - y[b, t, :, j] * s
                out[b, t, :, j] = y[b, t, :, i] * s + y[b, t, :, j] * c
    return out


def tree_sees(mask, t, s):
    """Whether drafted token t sees drafted token s; mask None: s <= t."""
    return s <= t if mask is None else bool((int(mask[t]) >> s) & 1)


def tree_attention(q, K, V, vis, n_vis, n_text, mask, scale):
    """One sequence: q [T][H][d]; K, V logical [Hkv][>= n_vis + n_text + T][d],
    the T tokens' own rows behind the text; vis [Hkv][k] or None; mask [T] bit
    sets or None.  Returns (out [T][H][d], lse [T][H], mag [T][H][d]); mag is
    the same average over |V|, which error bounds are relative to."""
    q, K, V = (np.asarray(a, dtype=np.float64) for a in (q, K, V))
    T, H, d = q.shape
    G = H // K.shape[0]
    out, lse, mag = np.zeros((T, H, d)), np.full((T, H), -math.inf), np.zeros((T, H, d))
    for t in range(T):
        drafted = [n_vis + n_text + s for s in range(T) if tree_sees(mask, t, s)]
        for h in range(H):
            g = h // G
            sel = range(n_vis) if vis is None else vis[g]
            tokens = np.array([int(i) for i in sel] + list(range(n_vis, n_vis + n_text)) + drafted, dtype=np.int64)
            if len(tokens) == 0:
                continue
            z = scale * (K[g, tokens] @ q[t, h])
            m = z.max()
            w = np.exp(z - m)
            out[t, h] = (w / w.sum()) @ V[g, tokens]
            mag[t, h] = (w / w.sum()) @ np.abs(V[g, tokens])
            lse[t, h] = m + math.log(w.sum())
    return out, lse, mag


def accept_path(X, base, path):
    """Logical rows X [..][tokens][d] with row base + path[i] at base + i."""
    X = np.array(X)
    old = X.copy()
    for i, p in enumerate(path):
        X[..., base + i, :] = old[..., base + int(p), :]
    return X


class PageBook:
    """Reference counts, tables and held pages, one entry at a time.  `ok` is
    False after a reservation that found too few free pages (and did nothing);
    `copies` lists the (shared page, private page) pairs of the last one."""

    def __init__(self, ref, table, n_pages):
        self.ref, self.n = [int(x) for x in ref], [int(x) for x in n_pages]
        self.table = [[int(x) for x in row] for row in table]
        self.ok, self.copies = True, []

    def release(self, keep):
        for b in range(len(self.n)):
            if keep[b] < 0:
                continue
            stay = min(self.n[b], -(-keep[b] // PAGE))
            for i in range(stay, self.n[b]):
                self.ref[self.table[b][i]] -= 1
                self.table[b][i] = -1
            self.n[b] = stay

    def fork(self, parent, child, n_tok=None):
        for i, (p, c) in enumerate(zip(parent, child)):
            take = self.n[p] if n_tok is None else -(-n_tok[i] // PAGE)
            for j in range(take):
                self.table[c][j] = self.table[p][j]
                self.ref[self.table[p][j]] += 1
            self.n[c] = take

    def reserve(self, length, new):
        want, before = [], list(self.ref)
        for b in range(len(self.n)):
            if new[b] == 0:
                continue
            first, last = length[b] // PAGE, (length[b] + new[b] - 1) // PAGE
            for i in range(min(first, self.n[b]), last + 1):
                if i >= self.n[b]:
                    want.append((b, i, -1))
                elif i >= first and before[self.table[b][i]] > 1:
                    want.append((b, i, self.table[b][i]))
        free = [p for p, r in enumerate(before) if r == 0]
        self.copies, self.ok = [], len(free) >= len(want)
        if not self.ok:
            return
        for (b, i, shared), page in zip(want, free):
            if shared >= 0:
                self.ref[shared] -= 1
                self.copies.append((shared, page))
            self.table[b][i] = page
            self.ref[page] = 1
            self.n[b] = max(self.n[b], i + 1)
